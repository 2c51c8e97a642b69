// The passes around the gated product of gemm_big.hip: T's planes, the gradients of G and U from
// dH (mx8.h), and what the adapter's gradients (grads8.hip) multiply.
//
//   dG = dH U sig (1 + G (1 - sig)), dU = dH G sig, sig = 1 / (1 + e^-G)     (glu.h)
//   Gr = s dZ L2^T, dL1 = X^T Gr, dL2 = s T^T dZ       for dZ = dG and dU (or a linear's dY)
//
// dL1 and dL2 are fp32, so what enters them is kept to 24 bits: dZ and Gr as three bf16
// planes whose sum they are (each takes what the ones before it rounded off).  dZ's planes
// exist on chip alone: the pass that forms Gr (k_glu_back) writes the first one, which is
// what the dX product takes, and the pass that forms dL2 (grads8.hip) computes dZ again from the
// 4 bytes an element that it came from.
#include <algorithm>

#include "glu.h"
#include "kernels.h"
#include "mx8.h"

namespace {

constexpr int kT = 256;
constexpr uint32_t kOOB = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
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

// ---- Gr's planes ---------------------------------------------------------------------
// The slices of Gr summed in order, scaled: bf16 [halves][M][r] and three planes [halves][3][M][rp]; and,
// where r is not its pitch rp, T with that pitch.  kN columns a thread (16-byte loads if 4).
template <int kN>
__global__ __launch_bounds__(kT) void k_low(Low q, int halves, int64_t M, int r, int rp) {
  const int h = blockIdx.y;
  const bool is_t = blockIdx.z == 1;
  const int64_t pitch = (int64_t)halves * M * r, n = M * rp;
  for (int64_t i = kN * ((int64_t)blockIdx.x * kT + threadIdx.x); i < n; i += (int64_t)kN * gridDim.x * kT) {
    const int64_t m = i / rp;
    const int c = (int)(i - m * rp);
    const int64_t at = ((int64_t)h * M + m) * r + c;
    if (is_t) {
#pragma unroll
      for (int j = 0; j < kN; ++j) q.Tp[h * n + i + j] = c + j < r ? q.T[at + j] : 0;
      continue;
    }
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
        if (a == 0 && c < r) q.G[at + j] = b[j];
      }
      uint16_t* to = q.planes + ((int64_t)h * 3 + a) * n + i;
      if constexpr (kN == 4) *(u32x2*)to = u32x2{b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16};
      else to[0] = b[0];
    }
  }
}

// ---- dZ and the slices of dZ L2^T ----------------------------------------------------
// Work group: 128 rows, eight waves of 16, and a slice of the columns in steps of 64.  Lane
// (x, q) holds row x, columns 16 q .. + 15 of a step: two matrix operands as they are, since a
// product may take the reduction in any order that both sides share.  The step's columns of L2
// (both halves) pass through LDS, two buffers; everything is loaded a step ahead.
constexpr int kBW = 8;                     // waves
constexpr int kBC = 64;                    // columns of a step
constexpr int kBPitch = kBC + 8;           // LDS row of L2: 16 rows' pieces of 16 bytes on different banks

// Eight elements from element c of a row of `cols` on, zeros past its end, whose first is `row` bytes into rs: a
// piece that crosses the end is read as the row's last eight and moved (one by one in rows of fewer).
__device__ __forceinline__ u32x4 load8(__amdgpu_buffer_rsrc_t rs, uint32_t row, int c, int cols, bool on) {
  const bool in = on && c < cols;
  if (cols >= 8) {                         // uniform
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, in ? row + 2 * min(c, cols - 8) : kOOB, 0, 0);
    return (cols & 7) == 0 || c + 8 <= cols ? v : qk::drop_front8(v, min(8, c + 8 - cols));
  }
  uint32_t e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    e[j] = __builtin_amdgcn_raw_buffer_load_b16(rs, in && c + j < cols ? row + 2 * (c + j) : kOOB, 0, 0);
  return u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
}

__global__ __launch_bounds__(64 * kBW, 4) void k_glu_back(const uint16_t* __restrict__ dH, int M, int F,
                                                          const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales,
                                                          const uint16_t* __restrict__ L2, int r, int chunk, int ldz,
                                                          uint16_t* __restrict__ dZ, float* __restrict__ part) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[2][2 * 64 * kBPitch];
  const int t = threadIdx.x, w = t >> 6, l = t & 63, x = l & 15, q = l >> 4;
  const int m = 16 * kBW * (int)blockIdx.x + 16 * w + x;
  const int f_beg = (int)blockIdx.y * chunk, f_end = min(F, f_beg + chunk);
  const int fp = (F + 31) / 32 * 32, nb = fp / 32;
  const bool ok = m < M;
  // all below 2^31 bytes; the up half's codes and scales follow the gate's
  const __amdgpu_buffer_rsrc_t rc = rsrc(codes, (uint64_t)2 * M * fp), rs = rsrc(scales, (uint64_t)2 * M * nb),
                               rd = rsrc(dH, (uint64_t)M * F * 2);
  const uint32_t up_c = (uint32_t)M * fp, up_s = (uint32_t)M * nb;
  const int nt = (r + 15) / 16, rk = 16 * nt;
  // L2's share of a thread: row lr of both halves, columns 8 lq .. + 7 of a step
  const int lr = t >> 3, lq = t & 7;
  f32x4 acc[2][4] = {};
  struct Step {
    u32x4 g, u, d[2], b[2];
    uint32_t sg, su;
  };
  auto load = [&](int f0) {
    Step s;
    const int f = f0 + 16 * q;
    const bool in = ok && f < f_end;       // rows of codes go on to a multiple of 32
    const uint32_t oc = in ? (uint32_t)m * fp + f : kOOB, os = in ? (uint32_t)m * nb + (f >> 5) : kOOB;
    s.g = __builtin_amdgcn_raw_buffer_load_b128(rc, oc, 0, 0);
    s.u = __builtin_amdgcn_raw_buffer_load_b128(rc, in ? oc + up_c : kOOB, 0, 0);
    s.sg = __builtin_amdgcn_raw_buffer_load_b8(rs, os, 0, 0);
    s.su = __builtin_amdgcn_raw_buffer_load_b8(rs, in ? os + up_s : kOOB, 0, 0);
    s.d[0] = load8(rd, (uint32_t)m * F * 2u, f, F, in);
    s.d[1] = load8(rd, (uint32_t)m * F * 2u, f + 8, F, in);
    const int fb = f0 + 8 * lq;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      s.b[h] = lr < r && fb < f_end ? qk::load8_row(L2 + ((int64_t)h * r + lr) * F, fb, F) : u32x4{0, 0, 0, 0};
    return s;
  };
  auto stage = [&](const Step& s, int buf) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (lr < rk) *(LDS_AS u32x4*)((LDS_AS uint16_t*)lds[buf] + (64 * h + lr) * kBPitch + 8 * lq) = s.b[h];
  };
  Step cur = load(f_beg);
  stage(cur, 0);
  int buf = 0;
  for (int f0 = f_beg; f0 < f_end; f0 += kBC, buf ^= 1) {
    const Step nxt = load(f0 + kBC);
    __syncthreads();                       // this step's L2 is in LDS, and the last one's reads are done
    const LDS_AS uint16_t* b2 = (const LDS_AS uint16_t*)lds[buf];
    const float ks = mx8::scale_f32(cur.sg), ku = mx8::scale_f32(cur.su);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int f = f0 + 16 * q + 8 * u;
      float dz[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float g[4], v[4];
        mx8::decode4(cur.g[2 * u + k], ks, g);
        mx8::decode4(cur.u[2 * u + k], ku, v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          glu::back(g[j], v[j], __uint_as_float(j & 1 ? cur.d[u][2 * k + (j >> 1)] & 0xFFFF0000u : cur.d[u][2 * k + (j >> 1)] << 16),
                    dz[0][4 * k + j], dz[1][4 * k + j]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < nt) b[j] = *(const LDS_AS u32x4*)(b2 + (64 * h + 16 * j + x) * kBPitch + 16 * q + 8 * u);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
          const u32x4 a = glu::take_plane(dz[h]);
          if (n == 0 && ok && f < F) qk::store8_row(dZ + (int64_t)m * ldz + h * F + f, a, min(8, F - f));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < nt) acc[h][j] = mfma16(a, b[j], acc[h][j]);
        }
      }
    }
    stage(nxt, buf ^ 1);
    cur = nxt;
  }
  if (f_end == F && ok && q == 0)
    for (int f = 2 * F; f < ldz; ++f) dZ[(int64_t)m * ldz + f] = 0;
  // lane: column 16 j + x, rows 4 q + v
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int mm = 16 * kBW * (int)blockIdx.x + 16 * w + 4 * q + v;
        const int c = 16 * j + x;
        if (mm < M && c < r) part[(((int64_t)blockIdx.y * 2 + h) * M + mm) * r + c] = acc[h][j][v];
      }
}

// Slices of that pass: about 512 work groups, of 128 columns at least.
struct PlanBack {
  int tiles, slices;
  int64_t chunk;
};
PlanBack plan_back(int64_t M, int64_t F) {
  PlanBack p;
  p.tiles = (int)((M + 16 * kBW - 1) / (16 * kBW));
  int64_t s = std::max<int64_t>(1, std::min<int64_t>(512 / p.tiles, F / 128));
  p.chunk = ((F + s - 1) / s + kBC - 1) / kBC * kBC;
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
  const unsigned z = rp == r ? 1 : 2;
  if (r % 4 == 0)
    hipLaunchKernelGGL(k_low<4>, dim3(blocks(M * rp / 4), (unsigned)halves, z), dim3(kT), 0, s, q, halves, M, r, rp);
  else
    hipLaunchKernelGGL(k_low<1>, dim3(blocks(M * rp), (unsigned)halves, z), dim3(kT), 0, s, q, halves, M, r, rp);
  return hipGetLastError();
}

size_t glu_back_ws(int64_t M, int64_t F, int r) { return (size_t)plan_back(M, F).slices * 2 * M * r * sizeof(float); }

hipError_t launch_glu_back(const uint16_t* dH, int64_t M, int64_t F, const uint8_t* gu_codes, const uint8_t* gu_scales,
                           const uint16_t* L2, int r, uint16_t* dZ, float* part, int* slices, hipStream_t s) {
  const PlanBack p = plan_back(M, F);
  *slices = p.slices;
  hipLaunchKernelGGL(k_glu_back, dim3((unsigned)p.tiles, (unsigned)p.slices), dim3(64 * kBW), 0, s, dH, (int)M, (int)F,
                     gu_codes, gu_scales, L2, r, (int)p.chunk, (int)glu_ldz(F), dZ, part);
  return hipGetLastError();
}
