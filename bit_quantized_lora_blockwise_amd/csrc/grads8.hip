// The adapter's gradients from activations kept in 8 bits, all in one launch:
//   dL1 = X^T Gr      [K, r]   X packed (mx8.h), Gr as three bf16 planes (24 bits); for each half of
//                              a gated product its own Gr
//   dL2 = s T^T dZ    [r, N]   dZ = dY as it is, or, for a gated product, dG and dU formed
//                              again in fp32 from dH and the packed G and U (glu.h)
// 4096 rows, r = 64: gated 4096 -> 2 x 11008 88 us (200 MB, 39 us at a copy's rate; dZ formed again keeps the
// vector units busy for 45, the planes' products the matrix units for 19, and a step's two phases overlap in
// part), a linear's 11008 -> 4096 39 us (79 MB, 15 us).
// Products that reduce over the long dimension M.  Work groups of eight waves take a slice of M
// in steps: the operands are loaded a step ahead into registers in row-major pieces of 16
// bytes, turned into bf16 on the way to LDS (dZ into three planes) and read back turned
// (ds_read_b64_tr_b16).  One LDS buffer and two barriers a step, so that two work groups share
// a CU and one converts while the other multiplies.  Slices are summed in order by
// k_grads8_sum, so results repeat.
//
// k_packed, k_dense: 256 columns, 64 rows a step; wave w takes 64 columns (w % 4) and half of
// the rows (w / 4).  k_gated: 128 columns, 32 rows a step, both halves; wave w takes 32 columns
// (w % 4) of half w / 4.
#include <algorithm>

#include "glu.h"
#include "kernels.h"
#include "mx8.h"

namespace {

constexpr int kT = 512;
constexpr int kP = 256, kM = 64;           // packed and dense
constexpr int kGP = 128, kGM = 32;         // gated
constexpr int kPitchB = 72;                // [m][c] tiles
constexpr int kABytes = kM * kP * 2;
constexpr int kBBytes = kM * kPitchB * 2;
constexpr int kGABytes = kGM * kGP * 2;    // of a plane of a half
constexpr int kGBBytes = kGM * kPitchB * 2;
constexpr int kLds = kABytes + 3 * kBBytes;
static_assert(6 * kGABytes + 2 * kGBBytes <= kLds, "the gated step fits");

using glu::kOOB;
using glu::rsrc;

enum Kind { kPacked, kDense, kGated };

struct Job {
  const uint8_t* codes;     // kPacked: X; kGated: G over U
  const uint8_t* scales;
  const uint16_t* d;        // kDense: dY; kGated: dH
  const uint16_t* B;        // kPacked: [planes][M][rp]; kDense: [M][r]; kGated: [2][M][r]
  int P, tiles, slices;
  int rows;                 // of a slice, a multiple of kM
  float* out;               // [slices] of P r (kGated: 2 P r) values
  float scale;
};

// A tiles [m][columns], 16-byte piece c of row m in slot c ^ 4 (m % 4), so that the rows that a transposed read
// touches fall on different banks.
template <int kRowBytes>
__device__ __forceinline__ int slot(int row, int piece) { return row * kRowBytes + 16 * (piece ^ (4 * (row & 3))); }

template <int kRowBytes>
__device__ __forceinline__ bf16x8 frag_a(const LDS_AS uint8_t* a, int m0, int p0) {
  const int l = threadIdx.x & 63, G = l >> 4, i = l & 15;
  const int row = m0 + ((G >> 1) << 3) + (i >> 2), p = p0 + ((G & 1) << 4) + ((i & 3) << 2);
  const LDS_AS uint8_t* at = a + slot<kRowBytes>(row, p >> 3) + 2 * (p & 7);
  const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4*)at);
  const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4*)(at + 4 * kRowBytes));
  const u32x2 u = __builtin_bit_cast(u32x2, x), v = __builtin_bit_cast(u32x2, y);
  return __builtin_bit_cast(bf16x8, u32x4{u[0], u[1], v[0], v[1]});
}

// kVec (dense): rows of d in whole 16-byte pieces.
template <Kind kKind, bool kVec, bool kVecR>
__device__ __forceinline__ void columns(const Job& jb, int M, int r, int rp, int tile, int slice, LDS_AS uint8_t* lds) {
  constexpr int kPlanes = kKind == kPacked ? 3 : 1;
  constexpr int kPieces = kKind == kPacked ? 2 : 4;
  const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63;
  const int wp = w & 3, wk = w >> 2;
  const int p0 = tile * kP, m_beg = slice * jb.rows, m_end = min(M, m_beg + jb.rows);
  const int cp = (jb.P + 31) / 32 * 32, nb = cp / 32;
  const __amdgpu_buffer_rsrc_t ra = kKind == kPacked ? rsrc(jb.codes, (uint64_t)M * cp) : rsrc(jb.d, (uint64_t)M * jb.P * 2);
  const __amdgpu_buffer_rsrc_t rs = rsrc(jb.scales, kKind == kPacked ? (uint64_t)M * nb : 0);
  __amdgpu_buffer_rsrc_t rb[kPlanes];      // one plane stays below 2^31 bytes, all together need not
#pragma unroll
  for (int j = 0; j < kPlanes; ++j) rb[j] = rsrc(jb.B + (int64_t)j * M * rp, (uint64_t)M * (kKind == kPacked ? rp : r) * 2);
  const int brow = t >> 3, bc = t & 7;
  struct Regs {
    u32x4 a[kPieces], b[kPlanes];
    uint32_t s[kPieces];
  };
  auto load = [&](int m) {
    Regs g;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if constexpr (kKind == kPacked) {    // rows t / 16 + 32 i, columns 16 (t % 16)
        const int row = m + (t >> 4) + 32 * i, p = p0 + 16 * (t & 15);
        const bool in = row < m_end && p < cp;
        g.a[i] = __builtin_amdgcn_raw_buffer_load_b128(ra, in ? (uint32_t)row * cp + p : kOOB, 0, 0);
        g.s[i] = __builtin_amdgcn_raw_buffer_load_b8(rs, in ? (uint32_t)row * nb + (p >> 5) : kOOB, 0, 0);
      } else {                             // rows t / 32 + 16 i, columns 8 (t % 32)
        const int row = m + (t >> 5) + 16 * i;
        g.a[i] = glu::load8<kVec>(ra, (uint32_t)row * jb.P * 2u, p0 + 8 * (t & 31), jb.P, row < m_end);
      }
    }
#pragma unroll
    for (int j = 0; j < kPlanes; ++j) {
      if constexpr (kKind == kPacked)
        g.b[j] = __builtin_amdgcn_raw_buffer_load_b128(
            rb[j], m + brow < m_end && 8 * bc < rp ? (uint32_t)((m + brow) * rp + 8 * bc) * 2u : kOOB, 0, 0);
      else g.b[j] = glu::load8<kVecR>(rb[j], 2u * (uint32_t)((m + brow) * r), 8 * bc, r, m + brow < m_end);
    }
    return g;
  };
  auto store = [&](const Regs& g) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if constexpr (kKind == kPacked) {
        const float s = mx8::scale_f32(g.s[i]);
        const int row = (t >> 4) + 32 * i;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v[8];
          mx8::decode4(g.a[i][2 * k], s, v);
          mx8::decode4(g.a[i][2 * k + 1], s, v + 4);
          *(LDS_AS u32x4*)(lds + slot<2 * kP>(row, 2 * (t & 15) + k)) =
              u32x4{qk::pack_bf16x2(v[0], v[1]), qk::pack_bf16x2(v[2], v[3]), qk::pack_bf16x2(v[4], v[5]),
                    qk::pack_bf16x2(v[6], v[7])};
        }
      } else {
        *(LDS_AS u32x4*)(lds + slot<2 * kP>((t >> 5) + 16 * i, t & 31)) = glu::fit8<kVec>(g.a[i], p0 + 8 * (t & 31), jb.P);
      }
    }
#pragma unroll
    for (int j = 0; j < kPlanes; ++j) *(LDS_AS u32x4*)(lds + kABytes + j * kBBytes + brow * (kPitchB * 2) + 16 * bc) =
        kKind == kPacked ? g.b[j] : glu::fit8<kVecR>(g.b[j], 8 * bc, r);
  };
  f32x16 acc[2][2] = {};
  Regs g = load(m_beg);
  for (int m = m_beg; m < m_end; m += kM) {
    __syncthreads();                       // the last step has been read
    store(g);
    g = load(m + kM);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = 32 * wk + 16 * s;
      const bf16x8 x0 = frag_a<2 * kP>(lds, k, 64 * wp), x1 = frag_a<2 * kP>(lds, k, 64 * wp + 32);
#pragma unroll
      for (int j = 0; j < kPlanes; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (32 * c < r) {
            const bf16x8 y = qk::frag_kmajor((const LDS_AS uint16_t*)(lds + kABytes + j * kBBytes), kPitchB, k, 32 * c);
            if constexpr (kKind == kPacked) {        // rows p, columns c
              acc[0][c] = qk::mfma32(x0, y, acc[0][c]);
              acc[1][c] = qk::mfma32(x1, y, acc[1][c]);
            } else {                                 // rows c, columns p
              acc[0][c] = qk::mfma32(y, x0, acc[0][c]);
              acc[1][c] = qk::mfma32(y, x1, acc[1][c]);
            }
          }
    }
  }
  // the two halves of each step's rows, 64 columns of them a wave pair
  __syncthreads();
  LDS_AS float* red = (LDS_AS float*)lds + wp * 2048 + l;
  float* out = jb.out + (int64_t)slice * jb.P * r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i) __syncthreads();
    if (wk == 1)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) red[(16 * j + e) * 64] = acc[i][j][e];
    __syncthreads();
    if (wk == 0)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int a = qk::acc_row(e), b = qk::acc_col(), q = p0 + 64 * wp + 32 * i;
          const int p = q + (kKind == kPacked ? a : b), c = 32 * j + (kKind == kPacked ? b : a);
          if (p < jb.P && c < r)
            out[kKind == kPacked ? (int64_t)p * r + c : (int64_t)c * jb.P + p] = jb.scale * (acc[i][j][e] + red[(16 * j + e) * 64]);
        }
  }
}

template <bool kVec, bool kVecR>
__device__ __forceinline__ void gated(const Job& jb, int M, int r, int tile, int slice, LDS_AS uint8_t* lds) {
  const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63;
  const int wp = w & 3, wh = w >> 2;
  const int p0 = tile * kGP, m_beg = slice * jb.rows, m_end = min(M, m_beg + jb.rows);
  const int cp = (jb.P + 31) / 32 * 32, nb = cp / 32;
  const __amdgpu_buffer_rsrc_t rc = rsrc(jb.codes, (uint64_t)2 * M * cp), rs = rsrc(jb.scales, (uint64_t)2 * M * nb),
                               rd = rsrc(jb.d, (uint64_t)M * jb.P * 2);
  const uint32_t up_c = (uint32_t)M * cp, up_s = (uint32_t)M * nb;
  // thread t: row t / 16, columns 8 (t % 16); of T half t / 256, row t / 8 % 32, ranks 8 (t % 8)
  const int row = t >> 4, piece = t & 15, p = p0 + 8 * piece;
  const int bh = t >> 8, brow = (t >> 3) & 31, bc = t & 7;
  const __amdgpu_buffer_rsrc_t rb = rsrc(jb.B + (int64_t)__builtin_amdgcn_readfirstlane(bh) * M * r, (uint64_t)M * r * 2);
  struct Regs {
    u32x2 g, u;
    u32x4 d, b;
    uint32_t sg, su;
  };
  auto load = [&](int m0) {
    Regs s;
    const int m = m0 + row;
    const bool in = m < m_end && p < cp;
    const uint32_t oc = in ? (uint32_t)m * cp + p : kOOB, os = in ? (uint32_t)m * nb + (p >> 5) : kOOB;
    s.g = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rc, oc, 0, 0));
    s.u = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rc, in ? oc + up_c : kOOB, 0, 0));
    s.sg = __builtin_amdgcn_raw_buffer_load_b8(rs, os, 0, 0);
    s.su = __builtin_amdgcn_raw_buffer_load_b8(rs, in ? os + up_s : kOOB, 0, 0);
    s.d = glu::load8<kVec>(rd, (uint32_t)m * jb.P * 2u, p, jb.P, m < m_end);
    s.b = glu::load8<kVecR>(rb, 2u * (uint32_t)((m0 + brow) * r), 8 * bc, r, m0 + brow < m_end);
    return s;
  };
  auto store = [&](const Regs& s) {
    const float kg = mx8::scale_f32(s.sg), ku = mx8::scale_f32(s.su);
    const u32x4 d = glu::fit8<kVec>(s.d, p, jb.P);
    float dz[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float g[4], u[4];
      mx8::decode4(s.g[k], kg, g);
      mx8::decode4(s.u[k], ku, u);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        glu::back(g[j], u[j], __uint_as_float(j & 1 ? d[2 * k + (j >> 1)] & 0xFFFF0000u : d[2 * k + (j >> 1)] << 16),
                  dz[0][4 * k + j], dz[1][4 * k + j]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 3; ++n)
        *(LDS_AS u32x4*)(lds + (3 * h + n) * kGABytes + slot<2 * kGP>(row, piece)) = glu::take_plane(dz[h]);
    *(LDS_AS u32x4*)(lds + 6 * kGABytes + bh * kGBBytes + brow * (kPitchB * 2) + 16 * bc) = glu::fit8<kVecR>(s.b, 8 * bc, r);
  };
  f32x16 acc[2] = {};
  Regs g = load(m_beg);
  for (int m = m_beg; m < m_end; m += kGM) {
    __syncthreads();                       // the last step has been read
    store(g);
    g = load(m + kGM);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kGM; k += 16) {
      bf16x8 y[2];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        y[c] = qk::frag_kmajor((const LDS_AS uint16_t*)(lds + 6 * kGABytes + wh * kGBBytes), kPitchB, k, 32 * c);
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        const bf16x8 x = frag_a<2 * kGP>(lds + (3 * wh + n) * kGABytes, k, 32 * wp);
        acc[0] = qk::mfma32(y[0], x, acc[0]);
        if (r > 32) acc[1] = qk::mfma32(y[1], x, acc[1]);
      }
    }
  }
  float* out = jb.out + ((int64_t)slice * 2 + wh) * jb.P * r;
  const int q = p0 + 32 * wp + qk::acc_col();
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int c = 32 * j + qk::acc_row(e);
      if (q < jb.P && c < r) out[(int64_t)c * jb.P + q] = jb.scale * acc[j][e];
    }
}

// Work groups: dL1's tiles and slices (for a gated product of one half, then of the other), then dL2's.
template <bool kGlu, bool kVec, bool kVecR>
__global__ __launch_bounds__(kT, 4) void k_grads8(Job j0, Job j0u, Job j1, int M, int r, int rp) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
  const int n0 = j0.tiles * j0.slices;
  int b = (int)blockIdx.x;
  if (b < n0) return columns<kPacked, true, true>(j0, M, r, rp, b % j0.tiles, b / j0.tiles, (LDS_AS uint8_t*)lds);
  b -= n0;
  if constexpr (kGlu) {
    if (b < n0) return columns<kPacked, true, true>(j0u, M, r, rp, b % j0.tiles, b / j0.tiles, (LDS_AS uint8_t*)lds);
    b -= n0;
    gated<kVec, kVecR>(j1, M, r, b % j1.tiles, b / j1.tiles, (LDS_AS uint8_t*)lds);
  } else {
    columns<kDense, kVec, kVecR>(j1, M, r, rp, b % j1.tiles, b / j1.tiles, (LDS_AS uint8_t*)lds);
  }
}

// Up to three outputs as their slices' sums, added in order.
struct Sum {
  const float* part;
  float* out;
  int64_t n;
  int slices, blocks;
};

template <int kN>
__device__ __forceinline__ void sum_span(const Sum& s, int blk) {
  const int64_t n = s.n / kN;
  typedef float vec __attribute__((ext_vector_type(kN)));
  const vec* p = (const vec*)s.part;
  for (int64_t i = (int64_t)blk * 256 + threadIdx.x; i < n; i += (int64_t)s.blocks * 256) {
    vec u = p[i];
    int k = 1;
    for (; k + 3 <= s.slices; k += 3) {
      const vec a = p[k * n + i], b = p[(k + 1) * n + i], c = p[(k + 2) * n + i];
      u += a;
      u += b;
      u += c;
    }
    for (; k < s.slices; ++k) u += p[k * n + i];
    ((vec*)s.out)[i] = u;
  }
}

__global__ __launch_bounds__(256) void k_grads8_sum(Sum a, Sum b, Sum c) {
  int blk = (int)blockIdx.x;
  const bool first = blk < a.blocks, second = !first && blk < a.blocks + b.blocks;
  const Sum s = first ? a : second ? b : c;
  blk -= first ? 0 : second ? a.blocks : a.blocks + b.blocks;
  if (s.n % 4 == 0) sum_span<4>(s, blk);
  else sum_span<1>(s, blk);
}

// Slices of M in whole steps, for about `groups` work groups.
struct Plan {
  int tiles, slices, rows;
};
Plan plan(int64_t P, int width, int64_t M, int groups) {
  Plan p;
  p.tiles = (int)((P + width - 1) / width);
  const int64_t steps = (M + kM - 1) / kM;
  // Up to four steps stay in one slice: their sum would be a launch of its own.  A linear's whole
  // backward, us, cut / in one: 1024 -> 1024 100 rows 33 / 30, 256 rows 34 / 32; 512 rows (8 steps)
  // 33 / 38, 1024 rows (16) 42 / 56.
  const int64_t s = steps <= 4 ? 1 : std::max<int64_t>(1, std::min<int64_t>(groups / p.tiles, steps));
  const int64_t per = (steps + s - 1) / s;
  p.rows = (int)(per * kM);
  p.slices = (int)((steps + per - 1) / per);
  return p;
}
struct Plans {
  Plan x, z;
};
// Two work groups a CU in all, shared so that they end together: a half's dL1 against dL2 of both
// is K to 5 N (4096 x 4096 with 2 x 11008: 88 us; K to 3 N 99, K to 12 N 131).
Plans plans(int64_t M, int64_t K, int64_t N, int halves) {
  if (halves == 2) {
    const int gx = std::max(1, (int)(512.0 * K / (2.0 * K + 5.0 * N)));
    return Plans{plan(K, kP, M, gx), plan(N, kGP, M, std::max(1, 512 - 2 * gx))};
  }
  const double x = 1.5 * K, z = 1.0 * N;             // three planes against twice the bytes
  const int gx = std::max(1, (int)(512 * x / (x + z)));
  return Plans{plan(K, kP, M, gx), plan(N, kP, M, std::max(1, 512 - gx))};
}

}  // namespace

size_t grads8_ws(int64_t M, int64_t K, int64_t N, int halves, int r) {
  const Plans p = plans(M, K, N, halves);
  return (size_t)halves * r * sizeof(float) * (p.x.slices * K + p.z.slices * N) + 3 * 256;
}

hipError_t launch_grads8(const Grads8& g, int64_t M, int64_t K, int64_t N, int halves, int r, float* ws, hipStream_t s) {
  const Plans p = plans(M, K, N, halves);
  const int rp = g_pitch(r);
  const int64_t nx = K * r, nz = halves * N * r;
  auto up = [](int64_t n) { return (n + 63) / 64 * 64; };
  float* px[2] = {ws, ws + up(p.x.slices * nx)};
  float* pz = px[1] + (halves == 2 ? up(p.x.slices * nx) : 0);
  Job jx[2];
  for (int h = 0; h < 2; ++h)
    jx[h] = Job{g.x_codes, g.x_scales, nullptr, g.planes + (int64_t)h * 3 * M * rp, (int)K, p.x.tiles, p.x.slices, p.x.rows,
                p.x.slices > 1 ? px[h] : g.dL1 + h * nx, 1.0f};
  const Job jz{g.gu_codes, g.gu_scales, g.d, g.T, (int)N, p.z.tiles, p.z.slices, p.z.rows, p.z.slices > 1 ? pz : g.dL2, g.scale};
  const dim3 grid((unsigned)(halves * p.x.tiles * p.x.slices + p.z.tiles * p.z.slices));
#define QL_G8(G, V, R) hipLaunchKernelGGL((k_grads8<G, V, R>), grid, dim3(kT), 0, s, jx[0], jx[1], jz, (int)M, r, rp)
#define QL_G8V(G)                          \
  do {                                     \
    if (N % 8 == 0 && r % 8 == 0) QL_G8(G, true, true); \
    else if (N % 8 == 0) QL_G8(G, true, false);         \
    else if (r % 8 == 0) QL_G8(G, false, true);         \
    else QL_G8(G, false, false);           \
  } while (0)
  if (halves == 2) QL_G8V(true);
  else QL_G8V(false);
#undef QL_G8V
#undef QL_G8
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (p.x.slices == 1 && p.z.slices == 1)) return e;
  auto sum = [](const float* part, float* out, int64_t n, int slices) {
    return Sum{part, out, n, slices, slices > 1 ? (int)std::max<int64_t>(1, std::min<int64_t>((n / 4 + 255) / 256, 2048)) : 0};
  };
  const Sum a = sum(px[0], g.dL1, nx, p.x.slices), b = sum(px[1], g.dL1 + nx, nx, halves == 2 ? p.x.slices : 1),
            c = sum(pz, g.dL2, nz, p.z.slices);
  hipLaunchKernelGGL(k_grads8_sum, dim3((unsigned)(a.blocks + b.blocks + c.blocks)), dim3(256), 0, s, a, b, c);
  return hipGetLastError();
}
