// The microscaled layer for few rows (single tokens, decode batches, short prompts):
// two launches forward, three backward, each spread over the whole chip, since the
// time is launches and latency (and, for one token, the weight's bytes).
//   1. k_small_down: one pass over the activations [M, R] quantises them and forms
//      the skinny product with the adapter (T = (D o X) L1, or G = dY L2^T) as fp32
//      partial sums over slices of the reduction.
//   2. k_mx4_small: the product with the packed weight.  A work group takes 16 rows of
//      the weight and 16 kMG activation rows, its waves split the reduction, and their
//      sums meet in LDS; it also adds the slices of T (or G), multiplies the
//      adapter's second factor and stores.  The work groups of the first 16 rows
//      write T (or G's planes) out.
// One token 4096 -> 11008, rank 64: 3.9 us and 7.2 us (24 MB of packed weight at 3.3
// TB/s); 77 rows 1000 -> 777, rank 12: 4.3 and 5.0 us.  A call is then bound by its two
// launches on the host, 2.6 us each, and the binding.
#include "mx4.h"

#include "kernels.h"

namespace {

using namespace mx4;

// ---------------------------------------------------------------------------
// Work group (m tile of 16 rows, slice, column tile of 16): sixteen waves, wave w the
// blocks w, w + 16, ... of the slice.  The operands of the 16x16x32 instruction are in
// quantisation order already: lane l holds eight elements of row l % 16, a quarter
// of a block; its block's other quarters are 16, 32 and 48 lanes on.
constexpr int kDW = 16;                      // waves
constexpr int kDThreads = 64 * kDW;
constexpr int kMaxSlices = 8;

// Blocks of a slice: whole rounds of the waves.  About 64 work groups in all, but no
// more than kMaxSlices slices: the product's work groups each add them up.
int slice_blocks(int64_t M, int64_t blocks, int r) {
  const int64_t tiles = (M + 15) / 16 * ((r + 15) / 16);
  int64_t s = 64 / tiles;
  s = s < 1 ? 1 : (s > kMaxSlices ? kMaxSlices : s);
  return kDW * (int)((blocks + kDW * s - 1) / (kDW * s));
}

// Loads through buffer descriptors: an offset out of range reads as 0 with no branch,
// so that every load of a round is in flight before the first is used.
constexpr uint32_t kOOB = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}

// Elements k .. k + 7 of a row of `len` bf16 that begins at byte `row`, zeros past its
// end (all of them if !on).  kVec: 16-byte pieces; else a piece that crosses the end is
// read as the last eight of the row and moved.
template <bool kVec>
__device__ __forceinline__ u32x4 load8(__amdgpu_buffer_rsrc_t rs, uint32_t row, int k, int len, bool on) {
  const bool in = on && k < len;
  if (kVec) return __builtin_amdgcn_raw_buffer_load_b128(rs, in ? row + 2 * k : kOOB, 0, 0);
  if (len >= 8) {
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, in ? row + 2 * min(k, len - 8) : kOOB, 0, 0);
    return k + 8 <= len ? v : qk::drop_front8(v, min(8, k + 8 - len));
  }
  uint32_t e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    e[j] = __builtin_amdgcn_raw_buffer_load_b16(rs, on && k + j < len ? row + 2 * (k + j) : kOOB, 0, 0);
  return u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
}

// kBkr: B(k, c) = Bm[k][c] (L1 [R, r]), else Bm[c][k] (L2 [r, R]).  kQuant: also packs A.
// blocks: of the packed length (a multiple of four).  kPair: the launch's second half of column tiles is a second
// product's, B and the slices behind the first's.
template <bool kBkr, bool kVec, bool kDrop, bool kQuant, bool kPair = false>
__global__ __launch_bounds__(kDThreads) void k_small_down(const uint16_t* __restrict__ A, int M, int R,
                                                          const uint16_t* __restrict__ Bm, int r, int blocks,
                                                          int per_slice, drop::Params d, uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales, float* __restrict__ part,
                                                          float out_scale) {
  __shared__ f32x4 red[kDW * 64];
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63, g = l >> 4, x = l & 15;
  const int m = 16 * (int)blockIdx.x + x, slice = blockIdx.y;
  int ctile = blockIdx.z;
  if (kPair && ctile >= (int)gridDim.z / 2) {
    ctile -= (int)gridDim.z / 2;
    Bm += (int64_t)R * r;
    part += (int64_t)gridDim.y * M * r;
  }
  const int c = 16 * ctile + x;
  const __amdgpu_buffer_rsrc_t ra = rsrc(A, (uint64_t)M * R * 2), rb = rsrc(Bm, (uint64_t)R * r * 2);
  const int last = min(blocks, (slice + 1) * per_slice);
  f32x4 acc = {0, 0, 0, 0};
#pragma unroll 2
  for (int q = slice * per_slice + w; q < last; q += kDW) {
    const int k = 32 * q + 8 * g;
    u32x4 b;
    if constexpr (kBkr) {
      uint32_t e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        e[j] = __builtin_amdgcn_raw_buffer_load_b16(rb, k + j < R && c < r ? (uint32_t)((k + j) * r + c) * 2u : kOOB, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = e[2 * j] | e[2 * j + 1] << 16;
    } else {
      b = load8<kVec>(rb, (uint32_t)(c * R) * 2u, k, R, c < r);
    }
    u32x4 a = load8<kVec>(ra, (uint32_t)(m * R) * 2u, k, R, m < M);
    if (kQuant && blockIdx.z == 0) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max((a[j] << 16) & 0x7FFFFFFFu, a[j] & 0x7FFF0000u));
      const uint32_t sb = scale_byte(max_over_rows(top));
      if (m < M) {
        codes[((int64_t)q * M + m) * 4 + g] = sb == 255u ? 0u : encode8(a, scale_f32(sb));
        if (g == 0) scales[((int64_t)(q >> 2) * M + m) * 4 + (q & 3)] = (uint8_t)sb;
      }
    }
    if constexpr (kDrop) a = drop::mask8(a, d, (uint32_t)m, (uint32_t)(4 * q + g));
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0,
                                                  0);
  }
  red[threadIdx.x] = acc;
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int i = 1; i < kDW; ++i) acc += red[64 * i + l];
    // lane l holds rows 4 g .. + 3 of column c
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int mm = 16 * (int)blockIdx.x + 4 * g + j;
      if (mm < M && c < r) part[((int64_t)slice * M + mm) * r + c] = out_scale * acc[j];
    }
  }
}

// ---------------------------------------------------------------------------
// Work group: 16 kPG rows of the weight, 16 kMG activation rows.  Waves 0 .. kPW - 1
// take pieces w, w + kPW, ... of the reduction (kAhead of them in flight).  Two more
// waves for each 16 activation rows form the adapter term meanwhile, each half of the
// rank so that its loads are in flight together; the first of them adds the
// halves and the other waves' sums in order and stores.
constexpr int kPW = 8;

struct SmallArgs {
  const uint32_t *ac, *as;          // packed activations, M rows
  const uint32_t *bc, *bs;          // packed weight, P rows
  int M, P, words;
  const float* part;                // slices of T or G, [S][M][r]
  int S;
  float low_scale;                  // T = bf16(low_scale sum), G likewise
  uint16_t* low_out;                // T [M, r] (may be nullptr) or G's three planes
  int low_pitch;                    // of those planes
  const uint16_t* LB;               // L2 [r, P] (forward), L1 [P, r] (backward)
  int r;
  float scale;                      // forward: Y += scale (T L2)
  drop::Params d;                   // backward
  uint16_t* C;
};

// kMode: 1 forward, 2 backward, 3 backward with dropout.
template <int kMode, int kMG, int kPG>
__global__ __launch_bounds__(64 * (kPW + 2 * kMG), kMG == 1 ? 8 : 4) void k_mx4_small(SmallArgs a) {
  constexpr int kAhead = kMG * kPG >= 8 ? 2 : 4;
  __shared__ f32x4 red[kPW][kPG][kMG][64], half[kPG][kMG][64];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, g = l >> 4, x = l & 15;
  const int p0 = 16 * kPG * (int)blockIdx.x, m0 = 16 * kMG * (int)blockIdx.y;

  if (w < kPW) {
    f32x4 acc[kPG][kMG];
#pragma unroll
    for (int j = 0; j < kPG; ++j)
#pragma unroll
      for (int i = 0; i < kMG; ++i) acc[j][i] = f32x4{0, 0, 0, 0};
    for (int q0 = w; q0 < a.words; q0 += kPW * kAhead) {
      u32x4 b[kAhead][kPG], ca[kAhead][kMG];
      uint32_t sb[kAhead][kPG], sa[kAhead][kMG];
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        const int q = min(q0 + n * kPW, a.words - 1);
#pragma unroll
        for (int j = 0; j < kPG; ++j) {
          const int p = min(p0 + 16 * j + x, a.P - 1);
          b[n][j] = *(const u32x4*)(a.bc + ((4 * q + g) * (int64_t)a.P + p) * 4);
          sb[n][j] = a.bs[q * (int64_t)a.P + p];
        }
#pragma unroll
        for (int i = 0; i < kMG; ++i) {
          const int m = min(m0 + 16 * i + x, a.M - 1);
          ca[n][i] = *(const u32x4*)(a.ac + ((4 * q + g) * (int64_t)a.M + m) * 4);
          sa[n][i] = a.as[q * (int64_t)a.M + m];
        }
      }
#pragma unroll
      for (int n = 0; n < kAhead; ++n)
        if (q0 + n * kPW < a.words) {
#pragma unroll
          for (int j = 0; j < kPG; ++j)
#pragma unroll
            for (int i = 0; i < kMG; ++i)
              acc[j][i] = mfma16(b[n][j], sb[n][j] >> (8 * g), ca[n][i], sa[n][i] >> (8 * g), acc[j][i]);
        }
    }
#pragma unroll
    for (int j = 0; j < kPG; ++j)
#pragma unroll
      for (int i = 0; i < kMG; ++i) red[w][j][i][l] = acc[j][i];
    __syncthreads();
    return;
  }

  // ---- adapter term of activation rows m0 + 16 i .. +15, columns 32 s .. +31 of the rank
  const int i = (w - kPW) >> 1, s = (w - kPW) & 1;
  const int ml = m0 + 16 * i + x, c = 32 * s + 8 * g;
  uint32_t e[kPG][8];
  const __amdgpu_buffer_rsrc_t rl = rsrc(a.LB, (uint64_t)a.P * a.r * 2);
#pragma unroll
  for (int j = 0; j < kPG; ++j) {
    const int p = min(p0 + 16 * j + x, a.P - 1);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t at = 2u * (kMode == 1 ? (uint32_t)((c + k) * a.P + p) : (uint32_t)(p * a.r + c + k));
      e[j][k] = __builtin_amdgcn_raw_buffer_load_b16(rl, c + k < a.r ? at : kOOB, 0, 0);
    }
  }
  // sums over the slices, in order
  const int64_t plane = (int64_t)a.M * a.r;             // of the slices
  const __amdgpu_buffer_rsrc_t rp = rsrc(a.part, (uint64_t)a.S * plane * 4);
  const uint32_t at = 4u * (uint32_t)(min(ml, a.M - 1) * a.r + c);
  float sum[8];
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    u32x4 v[kMaxSlices];      // slices past the last read as zeros
#pragma unroll
    for (int n = 0; n < kMaxSlices; ++n)
      v[n] = __builtin_amdgcn_raw_buffer_load_b128(rp, n < a.S ? at + 4u * k : kOOB, (int)(n * plane * 4), 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float u = __uint_as_float(v[0][j]);
#pragma unroll
      for (int n = 1; n < kMaxSlices; ++n) u += __uint_as_float(v[n][j]);
      sum[k + j] = c + k + j < a.r ? a.low_scale * u : 0.0f;
    }
  }
  u32x4 fr;
#pragma unroll
  for (int k = 0; k < 4; ++k) fr[k] = qk::pack_bf16x2(sum[2 * k], sum[2 * k + 1]);
  f32x4 low[kPG];
#pragma unroll
  for (int j = 0; j < kPG; ++j) {
    u32x4 fl;
#pragma unroll
    for (int k = 0; k < 4; ++k) fl[k] = e[j][2 * k] | e[j][2 * k + 1] << 16;
    low[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fl), __builtin_bit_cast(bf16x8, fr),
                                                     f32x4{0, 0, 0, 0}, 0, 0, 0);
  }
  if (a.low_out && blockIdx.x == 0 && ml < a.M) {
    // T [M][r]; G's planes (k_skinny_reduce3) [3][M][pitch], zeros past the rank
    const int pitch = kMode == 1 ? a.r : a.low_pitch;
    const int64_t gp = (int64_t)a.M * pitch;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + k < pitch) {
        uint16_t* o = a.low_out + (int64_t)ml * pitch + c + k;
        uint16_t hi = qk::f32_to_bf16(sum[k]);
        o[0] = hi;
        if constexpr (kMode != 1) {
          const float rest = sum[k] - qk::bf16_to_f32(hi);
          hi = qk::f32_to_bf16(rest);
          o[gp] = hi;
          o[2 * gp] = qk::f32_to_bf16(rest - qk::bf16_to_f32(hi));
        }
      }
  }
  if (s == 1) {
#pragma unroll
    for (int j = 0; j < kPG; ++j) half[j][i][l] = low[j];
    __syncthreads();
    return;
  }
  uint32_t keep[kPG];
  if constexpr (kMode == 3) {
#pragma unroll
    for (int j = 0; j < kPG; ++j) {
      const int p = p0 + 16 * j + 4 * g;
      keep[j] = drop::bits8(a.d, (uint32_t)ml, (uint32_t)(p >> 3)) >> (p & 4);
    }
  }
  __syncthreads();
  if (ml >= a.M) return;
#pragma unroll
  for (int j = 0; j < kPG; ++j) {
    // lane l holds columns 4 g .. +3 (of these 16) of activation row ml
    f32x4 out = red[0][j][i][l];
#pragma unroll
    for (int n = 1; n < kPW; ++n) out += red[n][j][i][l];
    low[j] += half[j][i][l];
    if constexpr (kMode == 1) low[j] *= a.scale;
    if constexpr (kMode == 3) {
#pragma unroll
      for (int k = 0; k < 4; ++k) low[j][k] = (keep[j] >> k) & 1u ? a.d.scale * low[j][k] : 0.0f;
    }
    out += low[j];
    const int p = p0 + 16 * j + 4 * g;
    uint16_t* dst = a.C + (int64_t)ml * a.P + p;
    if ((a.P & 3) == 0) {
      if (p < a.P) *(u32x2*)dst = u32x2{qk::pack_bf16x2(out[0], out[1]), qk::pack_bf16x2(out[2], out[3])};
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (p + k < a.P) dst[k] = qk::f32_to_bf16(out[k]);
    }
  }
}

template <int kMode>
hipError_t launch_product(const SmallArgs& a, hipStream_t s) {
#define QL_SM(MG, PG)                                                                        \
  hipLaunchKernelGGL((k_mx4_small<kMode, MG, PG>),                                           \
                     dim3((unsigned)((a.P + 16 * PG - 1) / (16 * PG)), (unsigned)((a.M + 16 * MG - 1) / (16 * MG))), \
                     dim3(64 * (kPW + 2 * MG)), 0, s, a)
  if (a.M <= 16) QL_SM(1, 1);
  else if (a.M <= 32) QL_SM(2, 1);
  else QL_SM(4, 2);
#undef QL_SM
  return hipGetLastError();
}

template <bool kBkr>
hipError_t launch_down(const uint16_t* A, int64_t M, int64_t R, const uint16_t* Bm, int r, const drop::Params& d,
                       uint8_t* codes, uint8_t* scales, float* part, int* slices, hipStream_t s, float out_scale = 1.0f,
                       bool pair = false) {
  const int blocks = (int)(padded(R) / kBlock), per = slice_blocks(M, blocks, r);
  *slices = (blocks + per - 1) / per;
  const dim3 grid((unsigned)((M + 15) / 16), (unsigned)*slices, (unsigned)((r + 15) / 16 << (int)pair));
#define QL_SD(V, D, ...)                                                                                                  \
  hipLaunchKernelGGL((k_small_down<kBkr, V, D, __VA_ARGS__>), grid, dim3(kDThreads), 0, s, A, (int)M, (int)R, Bm, r, blocks, \
                     per, d, (uint32_t*)codes, scales, part, out_scale)
  const bool vec = (R % 8) == 0, drop = kBkr && d.cut != 0;
  if constexpr (kBkr) {
    if (drop) {
      if (codes) {
        if (vec) QL_SD(true, true, true);
        else QL_SD(false, true, true);
      } else {
        if (vec) QL_SD(true, true, false);
        else QL_SD(false, true, false);
      }
      return hipGetLastError();
    }
    if (pair) {                            // of rows of whole blocks of 64
      QL_SD(true, false, false, true);
      return hipGetLastError();
    }
  }
  if (codes) {
    if (vec) QL_SD(true, false, true);
    else QL_SD(false, false, true);
  } else {
    if (vec) QL_SD(true, false, false);
    else QL_SD(false, false, false);
  }
#undef QL_SD
  return hipGetLastError();
}

}  // namespace

// Few rows, or outputs that one round of work groups (64 rows, 32 columns, one a CU) covers; two
// rounds while the reduction and the rank are short.  Whole calls with dropout, us, here / with
// tiles of 128 x 128: one round: forward 128 rows 4096 -> 4096 rank 64 14 / 27, 11008 -> 4096 29 /
// 46, 512 rows 1024 -> 1024 9 / 18, backward 128 rows 4096 -> 4096 28 / 35, 11008 dY columns 43 / 37;
// two: forward 256 rows 4096 -> 4096 rank 16 18 / 26, rank 64 24 / 28, 11008 -> 4096 51 / 48, backward
// rank 16 27 / 36, rank 64 42 / 38, 11008 dY columns 74 / 40; 512 rows 4096 -> 4096 rank 64 36 / 30,
// 72 / 49.  Above 512 rows one round, up to a reduction of 8192: forward 4096 rows 4096 -> 64 23 /
// 35, 2048 rows 512 -> 256 10 / 18, 11008 -> 64 60 / 59; backward 39 / 52, 29 / 35, 85 / 79.
bool mx4_small_ok(int64_t M, int64_t P, int64_t R, int r) {
  const int64_t groups = (P + 31) / 32 * ((M + 63) / 64);
  return M <= 64 || (groups <= 256 && (M <= 512 || R <= 8192)) ||
         (M <= 512 && groups <= 512 && R * ((r + 15) / 16) <= 4096);
}

size_t mx4_small_ws(int64_t M, int r) { return (size_t)kMaxSlices * M * r * sizeof(float); }

hipError_t launch_mx4_small_fwd(const uint16_t* X, int64_t M, int64_t K, int64_t N, const uint8_t* bc, const uint8_t* bs,
                                const uint16_t* L1, const uint16_t* L2, int r, float scale, const drop::Params& d,
                                uint16_t* Y, uint16_t* T_out, uint8_t* ac, uint8_t* as, float* part, hipStream_t s) {
  int S = 0;
  hipError_t e = launch_down<true>(X, M, K, L1, r, d, ac, as, part, &S, s);
  if (e != hipSuccess) return e;
  return launch_product<1>(SmallArgs{(const uint32_t*)ac, (const uint32_t*)as, (const uint32_t*)bc, (const uint32_t*)bs,
                                     (int)M, (int)N, (int)(padded(K) / kPad), part, S, d.cut ? d.scale : 1.0f, T_out, r,
                                     L2, r, scale, drop::Params{}, Y},
                           s);
}

hipError_t launch_mx4_small_dx(const uint16_t* dY, int64_t M, int64_t K, int64_t N, const uint8_t* bc, const uint8_t* bs,
                               const uint16_t* L1, const uint16_t* L2, int r, float scale, const drop::Params& d,
                               uint16_t* dX, uint16_t* G, uint8_t* ac, uint8_t* as, float* part, hipStream_t s) {
  int S = 0;
  hipError_t e = launch_down<false>(dY, M, N, L2, r, drop::Params{}, ac, as, part, &S, s);
  if (e != hipSuccess) return e;
  const SmallArgs a{(const uint32_t*)ac, (const uint32_t*)as, (const uint32_t*)bc, (const uint32_t*)bs, (int)M, (int)K,
                    (int)(padded(N) / kPad), part, S, scale, G, g_pitch(r), L1, r, 1.0f, d, dX};
  return d.cut ? launch_product<3>(a, s) : launch_product<2>(a, s);
}

hipError_t launch_mx4_small_t(const uint16_t* X, int64_t M, int64_t K, const uint16_t* L1, int r, const drop::Params& d,
                              uint16_t* T, float* part, hipStream_t s) {
  int S = 0;
  hipError_t e = launch_down<true>(X, M, K, L1, r, d, nullptr, nullptr, part, &S, s);
  if (e != hipSuccess) return e;
  return launch_skinny_reduce(part, S, M * r, d.cut ? d.scale : 1.0f, T, s);
}

hipError_t launch_mx4_small_g(const uint16_t* dY, int64_t M, int64_t N, const uint16_t* L2, int r, float scale,
                              uint16_t* G, float* part, hipStream_t s) {
  int S = 0;
  hipError_t e = launch_down<false>(dY, M, N, L2, r, drop::Params{}, nullptr, nullptr, part, &S, s);
  if (e != hipSuccess) return e;
  return launch_skinny_reduce3(part, S, M, r, scale, GPlanes{G, nullptr}, s);
}

hipError_t launch_small_slices(const uint16_t* A, int64_t M, int64_t R, const uint16_t* B, bool b_is_kr, int r,
                               const drop::Params& d, float scale, float* part, int* slices, hipStream_t s, bool pair) {
  return b_is_kr ? launch_down<true>(A, M, R, B, r, d, nullptr, nullptr, part, slices, s, scale, pair)
                 : launch_down<false>(A, M, R, B, r, drop::Params{}, nullptr, nullptr, part, slices, s, scale);
}
