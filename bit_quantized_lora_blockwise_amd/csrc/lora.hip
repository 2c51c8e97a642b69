// Skinny products of the LoRA branch (rank r <= 64):
//   T = bf16(X L1)            (forward, and recomputation in the backward)
//   G = bf16(s dY L2^T)       (backward)
//   dL1 = fp32(X^T G)         (backward)
//   dL2 = fp32(s T^T dY)      (backward)
// Layer formula and gradient flow: nlp-lineage milestone page on QLoRA,
// section "The idea", notation paragraph (only L1 and L2 get gradients).
//
// All four are memory-bound passes over an [M, R] bf16 activation.  Each work
// group owns a 64-row tile of the long dimension and one slice of the
// reduction; slices write fp32 partials that a second kernel sums in a fixed
// order, so results are deterministic.  With dropout on the adapter's input (T and
// dL1 of D o X) the mask of philox.h is drawn where a thread holds eight elements
// of a row, between the load and the LDS store or the MFMA; its scale goes into
// the sum of the slices.  Within a slice the 64-wide steps are
// pipelined: the tiles of step st + 2 are loaded into registers while step st
// multiplies out of one LDS buffer and step st + 1's tiles go into the other.
#include <algorithm>

#include "kernels.h"
#include "mx4.h"
#include "philox.h"
#include "tpart.h"

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;
constexpr int kPitch = 72;  // 64 + 8 elements of padding per LDS row
constexpr uint32_t kOOB = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)(bytes < 0x7FFFFFFFull ? bytes : 0x7FFFFFFFull),
                                           0x00020000);
}

// A 64 x 64 bf16 tile of a row-major matrix held in registers: thread t holds
// rows (t / 8) + 32 i, columns 8 (t % 8) .. +8.
struct Tile {
  u32x4 v[2];
};

// How a tile is read: in aligned 16-byte pieces (ld and cols multiples of 8, base 16-byte
// aligned), in pieces at any element (rows of at least eight), as the piece that begins
// with the row and goes on into the next ones (dense rows of fewer than eight, eight
// elements in all or more), element by element, or that by 64-bit address (matrices past
// the 2^31 bytes that a buffer offset reaches).  Each operand by its own rows: T of 4096 x
// 11008 at rank 1 took 58 us with both by elements, 24 so.
enum Load { kPieces, kAnywhere, kShort, kElements, kFar };

// Tile of a matrix with `ld` elements per row, its first row at `base`, its first column
// c0; rows at or past `rows` and columns at or past `cols` read as zero.  Each thread
// issues two 16-byte buffer loads (or sixteen of one element), with no branch, so that
// the loads of later steps stay in flight.  kAnywhere: a piece that crosses the row's end
// is read as the last eight of the row and moved into place by fit_tile.  kShort: likewise
// with the last eight of the matrix; `lead` elements of it, eight if there are as many, lie
// before `base`.  `bytes`: extent of the matrix from `base`.
template <Load kHow>
__device__ __forceinline__ Tile load_tile(const uint16_t* base, int64_t c0, int64_t ld, int64_t rows, int64_t cols,
                                          uint64_t bytes, int lead = 0) {
  const int t = threadIdx.x;
  const int64_t cc = c0 + (t & 7) * 8;
  const __amdgpu_buffer_rsrc_t rs = kHow == kShort ? rsrc(base - lead, bytes + 2 * lead) : rsrc(base, bytes);
  Tile tl;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = (t >> 3) + 32 * i;
    if constexpr (kHow == kFar) {
      uint32_t e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = row < rows && cc + j < cols ? base[row * ld + cc + j] : 0;
      tl.v[i] = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
    } else if constexpr (kHow == kShort) {
      const int64_t at = lead + min(row * ld, (int64_t)(bytes / 2) - 8);
      tl.v[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, row < rows && cc < cols ? (uint32_t)(at * 2) : kOOB, 0, 0);
    } else if constexpr (kHow != kElements) {
      const int64_t at = row * ld + (kHow == kPieces ? cc : min(cc, cols - 8));
      tl.v[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, row < rows && cc < cols ? (uint32_t)(at * 2) : kOOB, 0, 0);
    } else {
      uint32_t e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        e[j] = __builtin_amdgcn_raw_buffer_load_b16(
            rs, row < rows && cc + j < cols ? (uint32_t)((row * ld + cc + j) * 2) : kOOB, 0, 0);
      tl.v[i] = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
    }
  }
  return tl;
}

// total (kShort): elements of the matrix from the tile's first on.
template <Load kHow>
__device__ __forceinline__ void fit_tile(Tile& tl, int64_t c0, int64_t cols, int64_t total = 0) {
  if constexpr (kHow == kAnywhere) {
    const int64_t over = c0 + (threadIdx.x & 7) * 8 + 8 - cols;
    const int s = (int)max((int64_t)0, min((int64_t)8, over));
#pragma unroll
    for (int i = 0; i < 2; ++i) tl.v[i] = qk::drop_front8(tl.v[i], s);
  }
  if constexpr (kHow == kShort) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t over = ((threadIdx.x >> 3) + 32 * i) * cols + 8 - total;
      tl.v[i] = qk::drop_front8(tl.v[i], (int)max((int64_t)0, min((int64_t)8, over)));
#pragma unroll
      for (int j = 0; j < 4; ++j) tl.v[i][j] &= cols > 2 * j + 1 ? 0xFFFFFFFFu : cols > 2 * j ? 0xFFFFu : 0u;
    }
  }
}

__device__ __forceinline__ void store_tile(const Tile& tl, LDS_AS uint16_t* dst) {
  const int t = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 2; ++i) *(LDS_AS u32x4*)(dst + ((t >> 3) + 32 * i) * kPitch + (t & 7) * 8) = tl.v[i];
}

// Zeroes the dropped elements of a tile whose element (0, 0) is (m0, k0), k0 a
// multiple of 8.
__device__ __forceinline__ void drop_tile(Tile& tl, const drop::Params& d, int64_t m0, int64_t k0) {
  const int t = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    tl.v[i] = drop::mask8(tl.v[i], d, (uint32_t)(m0 + (t >> 3) + 32 * i), (uint32_t)(k0 >> 3) + (t & 7));
}

// C[M, r] partial over one reduction slice: A [M, R] (row stride lda) times B, where
// B(k, c) = Bm[k * r + c] (kBkr, L1 [R, r]) or Bm[c * R + k] (!kBkr, L2 [r, R]).
// kDrop: of D o A, not scaled.
template <bool kBkr, Load kA, Load kB, bool kDrop = false>
__global__ __launch_bounds__(kThreads) void k_lora_skinny(const uint16_t* __restrict__ A, int64_t M, int64_t R,
                                                          int64_t lda, const uint16_t* __restrict__ Bm, int r,
                                                          int64_t chunk, float* __restrict__ part, drop::Params d) {
  __shared__ __attribute__((aligned(16))) uint16_t As[2][kTile * kPitch];
  __shared__ __attribute__((aligned(16))) uint16_t Bs[2][kTile * kPitch];
  const int w = threadIdx.x >> 6;
  const int wm = w & 1, wc = w >> 1;
  const int64_t m0 = (int64_t)blockIdx.x * kTile;
  const int split = blockIdx.y;
  const int64_t k_beg = split * chunk;
  const int64_t k_end = min(R, k_beg + chunk);
  const int64_t nsteps = (k_end - k_beg + kTile - 1) / kTile;
  auto tiles = [&](int64_t st, Tile& ta, Tile& tb) {
    const int64_t k0 = k_beg + st * kTile;
    const int64_t kl = k_end - k0;                     // columns of the slice left (<= 0: zeros)
    const int64_t k0c = kl > 0 ? k0 : 0;
    const int64_t ke = kl > 0 ? k_end : 0;             // past the slice: no columns
    ta = load_tile<kA>(A + m0 * lda, k0c, lda, M - m0, ke, (uint64_t)((M - m0) * lda) * 2);
    if (kBkr) tb = load_tile<kB>(Bm + k0c * r, 0, r, kl, r, (uint64_t)((R - k0c) * r) * 2, (int)min((int64_t)8, k0c * r));
    else tb = load_tile<kB>(Bm, k0c, R, r, ke, (uint64_t)(r * R) * 2);
  };
  auto store = [&](int64_t st, Tile& ta, Tile& tb) {
    const int64_t k0 = k_beg + st * kTile;
    fit_tile<kA>(ta, k0, k_end);
    if (kBkr) fit_tile<kB>(tb, 0, r, (R - (k0 < k_end ? k0 : 0)) * r);
    else fit_tile<kB>(tb, k0, k_end);
    if constexpr (kDrop) drop_tile(ta, d, m0, k0);
    store_tile(ta, (LDS_AS uint16_t*)As[st & 1]);
    store_tile(tb, (LDS_AS uint16_t*)Bs[st & 1]);
  };
  f32x16 acc = {};
  auto step = [&](int64_t st, Tile& na, Tile& nb, Tile& la, Tile& lb) {
    tiles(st + 2, la, lb);
    const LDS_AS uint16_t* as = (const LDS_AS uint16_t*)As[st & 1];
    const LDS_AS uint16_t* bs = (const LDS_AS uint16_t*)Bs[st & 1];
    if (wc * 32 < r) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 a = qk::frag_rowmajor(as, kPitch, 32 * wm, 16 * s);
        bf16x8 b = kBkr ? qk::frag_kmajor(bs, kPitch, 16 * s, 32 * wc) : qk::frag_rowmajor(bs, kPitch, 32 * wc, 16 * s);
        acc = qk::mfma32(a, b, acc);
      }
    }
    store(st + 1, na, nb);
    __syncthreads();
  };
  Tile a0, b0, aA, bA, aB, bB;
  tiles(0, a0, b0);
  tiles(1, aA, bA);
  store(0, a0, b0);
  __syncthreads();
  for (int64_t st = 0; st < nsteps; st += 2) {   // an odd count runs one more step over zeros
    step(st, aA, bA, aB, bB);
    step(st + 1, aB, bB, aA, bA);
  }
  if (wc * 32 < r) {
    const int c = 32 * wc + qk::acc_col();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int64_t m = m0 + 32 * wm + qk::acc_row(j);
      if (m < M && c < r) part[((int64_t)split * M + m) * r + c] = acc[j];
    }
  }
}

// The same partial product for the common case (R, lda, r multiples of 8,
// 8 <= r <= 64, 16-byte aligned operands), laid out for streaming with about one
// work group per CU.  A work group owns 64 rows of A and one slice of the
// reduction and runs 16 waves: wave (g, p) takes rows 16 g .. 16 g + 15 of the
// tile, all r columns (four 16x16x32 MFMA tiles), and the 64-column steps
// p, p + 4, p + 8, ... of the slice.  The rows of A go straight from memory into
// MFMA operand registers (lane l: row l % 16, eight columns at 8 (l / 16)),
// kSkDepth of the wave's steps ahead; the four B tiles of a group of steps
// (64 x 64 each, from L2) are held in registers as far ahead and pass through
// double-buffered LDS, one barrier per group.
// At the end the four phases' sums are added in LDS in the order p = 0 .. 3.
// Per CU this keeps well over 100 KB of A in flight with four waves per SIMD,
// while each slice of B is read once per 64 rows and the slices stay few.
// kQuant: the pass also writes A in microscaled 4-bit (layout: mx4.h), which a pass of
// its own would read A again for (9.5 us at 2048 x 8192).  Lanes l, l + 16, l + 32 and
// l + 48 hold the four quarters of a block: its largest magnitude is two register
// swaps away, and each lane packs its own eight elements.
constexpr int kSkGroups = 4;                       // row groups of 16
constexpr int kSkPhases = 4;                       // steps taken in turn
constexpr int kSkThreads = 64 * kSkGroups * kSkPhases;
constexpr int kSkDepth = 4;                        // groups of A and B in flight

struct PackTo {
  uint32_t* codes;
  uint8_t* scales;
  int64_t padded;      // row length as packed, a multiple of 128
};

template <bool kBkr, bool kDrop = false, bool kQuant = false>
__global__ __launch_bounds__(kSkThreads, 1) void k_lora_skinny_stream(const uint16_t* __restrict__ A, int64_t M,
                                                                     int64_t R, int64_t lda,
                                                                     const uint16_t* __restrict__ Bm, int r,
                                                                     int64_t chunk, float* __restrict__ part,
                                                                     drop::Params d, PackTo to) {
  __shared__ __attribute__((aligned(16))) uint16_t Bs[2][kSkPhases][kTile * kPitch];
  const int t = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63;
  const int rg = w % kSkGroups, ph = w / kSkGroups;
  const int64_t m0 = (int64_t)blockIdx.x * kTile;
  const int split = blockIdx.y;
  const int64_t k_beg = split * chunk;
  const int64_t k_end = min(R, k_beg + chunk);
  // the last slice's steps go on to the end of the packed length, over zeros
  const int64_t k_pack = kQuant ? (k_end == R ? to.padded : k_end) : k_end;
  const int nsteps = (int)((k_pack - k_beg + kTile - 1) / kTile);
  const int ngroups = (nsteps + kSkPhases - 1) / kSkPhases;   // group gi: steps kSkPhases gi + p

  // A operand: lane l reads row m0 + 16 rg + l % 16, columns k + 8 (l / 16) .. +8
  const int64_t arow = m0 + 16 * rg + (l & 15);
  const __amdgpu_buffer_rsrc_t ra = rsrc(A, (uint64_t)M * lda * 2);
  const uint32_t abase = (uint32_t)(arow * lda * 2);
  const int64_t akq = 8 * (l >> 4);
  auto load_a = [&](int gi, u32x4 (&v)[2]) {
    const int64_t k0 = k_beg + (int64_t)(kSkPhases * gi + ph) * kTile;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t k = k0 + 32 * u + akq;
      const bool ok = arow < M && k < k_end;             // k_end is a multiple of 8
      v[u] = __builtin_amdgcn_raw_buffer_load_b128(ra, ok ? abase + (uint32_t)(k * 2) : kOOB, 0, 0);
    }
  };
  // B tiles of a group: threads 256 q .. 256 q + 255 move the tile of step
  // kSkPhases gi + q, thread tt row tt / 8 (+32), eight columns at 8 (tt % 8);
  // kBkr: tile [k][c] from L1 [R, r]; otherwise tile [c][k] from L2 [r, R]
  const __amdgpu_buffer_rsrc_t rb = rsrc(Bm, (uint64_t)R * r * 2);
  const int bq = t >> 8, tt = t & 255;
  auto load_b = [&](int gi, u32x4 (&v)[2]) {
    const int64_t k0 = k_beg + (int64_t)(kSkPhases * gi + bq) * kTile;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = (tt >> 3) + 32 * i, q = 8 * (tt & 7);
      bool ok;
      int64_t off;
      if (kBkr) {
        ok = k0 + rr < k_end && q < r;
        off = (k0 + rr) * r + q;
      } else {
        ok = rr < r && k0 + q < k_end;
        off = (int64_t)rr * R + k0 + q;
      }
      v[i] = __builtin_amdgcn_raw_buffer_load_b128(rb, ok ? (uint32_t)(off * 2) : kOOB, 0, 0);
    }
  };
  auto store_b = [&](const u32x4 (&v)[2], int buf) {
    LDS_AS uint16_t* dst = (LDS_AS uint16_t*)Bs[buf][bq];
#pragma unroll
    for (int i = 0; i < 2; ++i) *(LDS_AS u32x4*)(dst + ((tt >> 3) + 32 * i) * kPitch + 8 * (tt & 7)) = v[i];
  };
  // B operand of the 16x16x32 MFMA: lane l holds B(k + 8 (l / 16) .. +8, c + l % 16)
  auto frag_b = [&](const LDS_AS uint16_t* bs, int k, int c) -> bf16x8 {
    const int G = l >> 4, i = l & 15;
    if (kBkr) {
      // [k][c] tile: transposed reads, each 16-lane group a 4 x 16 block
      const LDS_AS uint16_t* p = bs + (k + 8 * G + (i >> 2)) * kPitch + c + 4 * (i & 3);
      i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4*)p);
      i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4*)(p + 4 * kPitch));
      u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
      return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
    }
    return *(const LDS_AS bf16x8*)(bs + (c + i) * kPitch + k + 8 * G);
  };

  // this wave's A rows and the work group's B tiles, kSkDepth groups ahead: group
  // gi's A in a[gi % kSkDepth], its B tiles in breg[gi % kSkDepth] until they are
  // stored to LDS during group gi - 1
  u32x4 a[kSkDepth][2], breg[kSkDepth][2];
  // Loads return in issue order, so the B tiles (small, soon needed) are
  // requested ahead of the A rows: a wait for a B tile then never waits for A.
  {
    u32x4 b0[2];
    load_b(0, b0);
#pragma unroll
    for (int j = 1; j <= kSkDepth; ++j) load_b(j, breg[j % kSkDepth]);
#pragma unroll
    for (int j = 0; j < kSkDepth; ++j) load_a(j, a[j]);
    store_b(b0, 0);
  }
  __syncthreads();
  f32x4 acc[4] = {};
  const int ntile = (r + 15) / 16;
  // group gi: MFMAs out of Bs[gi & 1], the tiles of gi + 1 into the other
  // buffer, then the tiles of gi + 1 + kSkDepth and this wave's A rows of
  // gi + kSkDepth are requested
  auto group = [&](int gi, u32x4 (&av)[2], u32x4 (&bn)[2]) {
    const LDS_AS uint16_t* bs = (const LDS_AS uint16_t*)Bs[gi & 1][ph];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if constexpr (kQuant) {
        const int64_t k = k_beg + (int64_t)(kSkPhases * gi + ph) * kTile + 32 * u;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max((av[u][j] << 16) & 0x7FFFFFFFu, av[u][j] & 0x7FFF0000u));
        const uint32_t sb = mx4::scale_byte(mx4::max_over_rows(top));
        if (arow < M && k < k_pack) {
          const int64_t blk = k >> 5;
          to.codes[(blk * M + arow) * 4 + (l >> 4)] = sb == 255u ? 0u : mx4::encode8(av[u], mx4::scale_f32(sb));
          if (l < 16) to.scales[((blk >> 2) * M + arow) * 4 + (blk & 3)] = (uint8_t)sb;
        }
      }
      if constexpr (kDrop) {
        const int64_t k = k_beg + (int64_t)(kSkPhases * gi + ph) * kTile + 32 * u + akq;
        av[u] = drop::mask8(av[u], d, (uint32_t)arow, (uint32_t)(k >> 3));
      }
      const bf16x8 x = __builtin_bit_cast(bf16x8, av[u]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < ntile) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, frag_b(bs, 32 * u, 16 * j), acc[j], 0, 0, 0);
    }
    store_b(bn, (gi + 1) & 1);
    load_b(gi + 1 + kSkDepth, bn);
    load_a(gi + kSkDepth, av);
    __syncthreads();
  };
  for (int g0 = 0; g0 < ngroups; g0 += kSkDepth) {
#pragma unroll
    for (int j = 0; j < kSkDepth; ++j)
      if (g0 + j < ngroups) group(g0 + j, a[j], breg[(j + 1) % kSkDepth]);
  }
  // the phases' sums added in order p = 0 .. 3 (the LDS tiles are free: every
  // wave has passed the barrier after its last fragment reads)
  float* red = (float*)&Bs[0][0][0];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) red[(w * 16 + 4 * j + v) * 64 + l] = acc[j][v];
  __syncthreads();
  if (ph == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = 16 * j + (l & 15);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float sum = red[(rg * 16 + 4 * j + v) * 64 + l];
#pragma unroll
        for (int p = 1; p < kSkPhases; ++p) sum += red[((p * kSkGroups + rg) * 16 + 4 * j + v) * 64 + l];
        // lane l holds C[4 (l / 16) + v][16 j + l % 16]
        const int64_t m = m0 + 16 * rg + 4 * (l >> 4) + v;
        if (j < ntile && m < M && c < r) part[((int64_t)split * M + m) * r + c] = sum;
      }
    }
  }
}

// Sum of `splits` fp32 partials, part[k * n + i], added in order k = 0, 1, ...
// starting from 0 (every path that adds these partials uses this order).
// Four outputs per thread: 16-byte loads, all splits' loads of a group of
// four issued before the additions.
__device__ __forceinline__ f32x4 sum_splits4(const f32x4* __restrict__ p4, int splits, int64_t n4, int64_t i4) {
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  int k = 0;
  for (; k + 4 <= splits; k += 4) {
    const f32x4 a = p4[(k + 0) * n4 + i4], b = p4[(k + 1) * n4 + i4];
    const f32x4 c = p4[(k + 2) * n4 + i4], d = p4[(k + 3) * n4 + i4];
    s += a;
    s += b;
    s += c;
    s += d;
  }
  for (; k < splits; ++k) s += p4[k * n4 + i4];
  return s;
}

__global__ __launch_bounds__(kThreads) void k_skinny_reduce(const float* __restrict__ part, int splits, int64_t n,
                                                            float scale, uint16_t* __restrict__ out) {
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  const int64_t t0 = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if ((n & 3) == 0) {
    const int64_t n4 = n >> 2;
    for (int64_t i4 = t0; i4 < n4; i4 += stride) {
      const f32x4 s = sum_splits4((const f32x4*)part, splits, n4, i4);
      *(u32x2*)(out + 4 * i4) = u32x2{qk::pack_bf16x2(scale * s[0], scale * s[1]),
                                      qk::pack_bf16x2(scale * s[2], scale * s[3])};
    }
    return;
  }
  for (int64_t i = t0; i < n; i += stride) {
    float s = 0.0f;
    for (int k = 0; k < splits; ++k) s += part[k * n + i];
    out[i] = qk::f32_to_bf16(scale * s);
  }
}

// The same sum kept to 24 bits as three bf16 planes [M][rp] (rp = r rounded up to 8,
// zeros past r) whose sum it is: each plane takes what the ones before it rounded
// off (exact in fp32), so a product with the planes loses nothing that fp32 would
// keep, while the first plane alone is the bf16 rounding.  Whole 16-byte pieces
// whatever r is: the planes are read again for every 64 columns of the activation.
// dense (rp != r): the first plane as [M][r] too.
__global__ __launch_bounds__(kThreads) void k_skinny_reduce3(const float* __restrict__ part, int splits, int64_t M, int r,
                                                             int rp, float scale, uint16_t* __restrict__ out,
                                                             uint16_t* __restrict__ dense) {
  const int64_t stride = (int64_t)gridDim.x * kThreads, n = M * rp;
  const int64_t t0 = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  for (int64_t i4 = t0; i4 < n / 4; i4 += stride) {
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    int64_t at = 0;
    int c = 0;
    if (r == rp) {
      x = scale * sum_splits4((const f32x4*)part, splits, n >> 2, i4);
    } else {
      const int64_t m = 4 * i4 / rp;
      c = (int)(4 * i4 - m * rp);
      at = m * r + c;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float s = 0.0f;
        if (c + j < r)
          for (int k = 0; k < splits; ++k) s += part[k * M * r + at + j];
        x[j] = scale * s;
      }
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const u32x2 h = {qk::pack_bf16x2(x[0], x[1]), qk::pack_bf16x2(x[2], x[3])};
      *(u32x2*)(out + j * n + 4 * i4) = h;
      if (j == 0 && dense) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < r) dense[at + e] = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
      }
      x -= f32x4{__uint_as_float(h[0] << 16), __uint_as_float(h[0] & 0xFFFF0000u), __uint_as_float(h[1] << 16),
                 __uint_as_float(h[1] & 0xFFFF0000u)};
    }
  }
}

// C[p, c] partial over one slice of m: sum_m A[m][p] * B[m][c], A [M, P], B [M, r];
// this work group's tile of 64 p is `tile`, its slice of m is `split`.  kDrop: of
// D o A, not scaled.  kPlanes: B is the sum of that many matrices, B + j M ldb.
// lds: (2 + 2 kPlanes) tiles of kTile * kPitch.  scale: of what is written; tr: written
// as part[c][p] (both for a product of one slice, whose partial is the result).
template <Load kA, Load kB, bool kDrop = false, int kPlanes = 1>
__device__ __forceinline__ void tn_tile(const uint16_t* __restrict__ A, int64_t lda, const uint16_t* __restrict__ B,
                                        int64_t M, int64_t P, int r, int64_t chunk, float* __restrict__ part,
                                        int tile, int split, uint16_t* lds, const drop::Params& d, int ldb,
                                        float scale = 1.0f, bool tr = false) {
  LDS_AS uint16_t* const sm = (LDS_AS uint16_t*)lds;
  auto abuf = [&](int64_t b) { return sm + (b & 1) * kTile * kPitch; };
  auto bbuf = [&](int64_t b, int j) { return sm + (2 + kPlanes * (b & 1) + j) * kTile * kPitch; };
  struct BTiles {
    Tile p[kPlanes];
  };
  const int w = threadIdx.x >> 6;
  const int wp = w & 1, wc = w >> 1;
  const int64_t p0 = (int64_t)tile * kTile;
  const int64_t m_beg = split * chunk;
  const int64_t m_end = min(M, m_beg + chunk);
  const int64_t nsteps = (m_end - m_beg + kTile - 1) / kTile;
  auto tiles = [&](int64_t st, Tile& ta, BTiles& tb) {
    const int64_t mm = m_beg + st * kTile;
    const int64_t ml = m_end - mm;                     // rows of the slice left (<= 0: zeros)
    const int64_t mmc = ml > 0 ? mm : 0;
    ta = load_tile<kA>(A + mmc * lda, p0, lda, ml, P, (uint64_t)((M - mmc) * lda) * 2);   // [m][p]
#pragma unroll
    for (int j = 0; j < kPlanes; ++j)
      tb.p[j] = load_tile<kB>(B + (j * M + mmc) * ldb, 0, ldb, ml, r, (uint64_t)((M - mmc) * ldb) * 2,
                              (int)min((int64_t)8, mmc * ldb));   // [m][c]
  };
  auto store = [&](int64_t st, Tile& ta, BTiles& tb) {
    fit_tile<kA>(ta, p0, P);
    if constexpr (kDrop) drop_tile(ta, d, m_beg + st * kTile, p0);
    store_tile(ta, abuf(st));
#pragma unroll
    for (int j = 0; j < kPlanes; ++j) {
      const int64_t mm = m_beg + st * kTile;
      fit_tile<kB>(tb.p[j], 0, r, (M - (mm < m_end ? mm : 0)) * ldb);
      store_tile(tb.p[j], bbuf(st, j));
    }
  };
  f32x16 acc = {};
  auto step = [&](int64_t st, Tile& na, BTiles& nb, Tile& la, BTiles& lb) {
    tiles(st + 2, la, lb);
    if (wc * 32 < r) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 a = qk::frag_kmajor(abuf(st), kPitch, 16 * s, 32 * wp);
#pragma unroll
        for (int j = 0; j < kPlanes; ++j)
          acc = qk::mfma32(a, qk::frag_kmajor(bbuf(st, j), kPitch, 16 * s, 32 * wc), acc);
      }
    }
    store(st + 1, na, nb);
    __syncthreads();
  };
  Tile a0, aA, aB;
  BTiles b0, bA, bB;
  tiles(0, a0, b0);
  tiles(1, aA, bA);
  store(0, a0, b0);
  __syncthreads();
  for (int64_t st = 0; st < nsteps; st += 2) {
    step(st, aA, bA, aB, bB);
    step(st + 1, aB, bB, aA, bA);
  }
  if (wc * 32 < r) {
    const int c = 32 * wc + qk::acc_col();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int64_t p = p0 + 32 * wp + qk::acc_row(j);
      if (p < P && c < r) part[tr ? c * P + p : ((int64_t)split * P + p) * r + c] = scale * acc[j];
    }
  }
}

template <Load kA, Load kB>
__global__ __launch_bounds__(kThreads) void k_lora_tn(const uint16_t* __restrict__ A, int64_t lda,
                                                      const uint16_t* __restrict__ B, int64_t M, int64_t P, int r,
                                                      int64_t chunk, float* __restrict__ part) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[4 * kTile * kPitch];
  tn_tile<kA, kB>(A, lda, B, M, P, r, chunk, part, blockIdx.x, blockIdx.y, lds, drop::Params{}, r);
}

// Two independent products of this kind in one launch (the backward's dL1 and
// dL2): work groups 0 .. n0 - 1 take the first, the rest the second.
struct TnJob {
  const uint16_t* A;
  int64_t lda;
  const uint16_t* B;
  int64_t P, chunk;
  float* part;
  int tiles, splits;
};

template <Load kA, Load kB>
__global__ __launch_bounds__(kThreads) void k_lora_tn_pair(TnJob j0, TnJob j1, int64_t M, int r) {
  const int n0 = j0.tiles * j0.splits;
  const bool second = (int)blockIdx.x >= n0;         // uniform over the work group
  const TnJob j = second ? j1 : j0;
  const int b = second ? (int)blockIdx.x - n0 : (int)blockIdx.x;
  __shared__ __attribute__((aligned(16))) uint16_t lds[4 * kTile * kPitch];
  tn_tile<kA, kB>(j.A, j.lda, j.B, M, j.P, r, j.chunk, j.part, b % j.tiles, b / j.tiles, lds, drop::Params{},
                        r);
}

// The pair with dropout on the first product's A and its B in three planes of pitch
// rp.  With one slice each, j0.part and j1.part are the results: scaled, the second
// transposed.  For what lora_grads.hip does not take (few rows, or sizes that are no
// multiples of 8): 130 rows of 520 and 333 columns, rank 5, 7.4 us; 4093 rows of 4097 and
// 11007, rank 37, 48 us (2.6 TB/s).
template <Load kA, Load kT, bool kDrop>
__global__ __launch_bounds__(kThreads) void k_lora_tn_pair3(TnJob j0, TnJob j1, int64_t M, int r, int rp,
                                                            drop::Params d, float scale0, float scale1, bool whole) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[8 * kTile * kPitch];
  const int n0 = j0.tiles * j0.splits;
  const int b = (int)blockIdx.x;
  if (b < n0)
    tn_tile<kA, kPieces, kDrop, 3>(j0.A, j0.lda, j0.B, M, j0.P, r, j0.chunk, j0.part, b % j0.tiles, b / j0.tiles, lds, d,
                                   rp, scale0);
  else
    tn_tile<kA, kT>(j1.A, j1.lda, j1.B, M, j1.P, r, j1.chunk, j1.part, (b - n0) % j1.tiles, (b - n0) / j1.tiles,
                          lds, d, r, scale1, whole);
}

// out[i] = scale * (sum of the slices), i over P * r, by work groups blk of nblk.
__device__ __forceinline__ void tn_reduce_span(const float* __restrict__ part, int splits, int64_t P, int r,
                                               float scale, float* __restrict__ out, int blk, int nblk) {
  const int64_t n = P * r;
  const int64_t stride = (int64_t)nblk * kThreads;
  const int64_t t0 = (int64_t)blk * kThreads + threadIdx.x;
  if ((n & 3) == 0) {
    const int64_t n4 = n >> 2;
    for (int64_t i4 = t0; i4 < n4; i4 += stride) ((f32x4*)out)[i4] = scale * sum_splits4((const f32x4*)part, splits, n4, i4);
    return;
  }
  for (int64_t i = t0; i < n; i += stride) {
    float s = 0.0f;
    for (int k = 0; k < splits; ++k) s += part[k * n + i];
    out[i] = scale * s;
  }
}

__global__ __launch_bounds__(kThreads) void k_tn_reduce(const float* __restrict__ part, int splits, int64_t P, int r,
                                                        float scale, float* __restrict__ out) {
  tn_reduce_span(part, splits, P, r, scale, out, blockIdx.x, gridDim.x);
}

// Same sum written transposed, out[c * P + p] for the partial element p * r + c:
// a work group takes 16 consecutive p, adds its 16 x r partials (each thread
// four adjacent c of one p when r % 4 == 0, all loads of a group issued
// together) into LDS and writes r rows of 16 contiguous outputs.
constexpr int kTrP = 16;

__device__ __forceinline__ void tn_reduce_t_block(const float* __restrict__ part, int splits, int64_t P, int r,
                                                  float scale, float* __restrict__ out, int blk) {
  __shared__ float tile[kTrP][65];
  const int64_t n = P * r;
  const int64_t p0 = (int64_t)blk * kTrP;
  const int np = (int)min((int64_t)kTrP, P - p0);
  if ((r & 3) == 0) {
    const int r4 = r >> 2;
    for (int e = threadIdx.x; e < np * r4; e += kThreads) {
      const int pl = e / r4, c4 = e - pl * r4;
      const f32x4 v = scale * sum_splits4((const f32x4*)part, splits, n >> 2, ((p0 + pl) * r >> 2) + c4);
#pragma unroll
      for (int j = 0; j < 4; ++j) tile[pl][4 * c4 + j] = v[j];
    }
  } else {
    for (int e = threadIdx.x; e < np * r; e += kThreads) {
      const int pl = e / r, c = e - pl * r;
      const int64_t i = (p0 + pl) * r + c;
      float s = 0.0f;
      for (int k = 0; k < splits; ++k) s += part[k * n + i];
      tile[pl][c] = scale * s;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < r * kTrP; e += kThreads) {
    const int c = e / kTrP, pl = e - c * kTrP;
    if (pl < np) out[(int64_t)c * P + p0 + pl] = tile[pl][c];
  }
}

__global__ __launch_bounds__(kThreads) void k_tn_reduce_t(const float* __restrict__ part, int splits, int64_t P, int r,
                                                          float scale, float* __restrict__ out) {
  tn_reduce_t_block(part, splits, P, r, scale, out, blockIdx.x);
}

// The two sums of a k_lora_tn_pair launch in one launch: work groups 0 .. nb0 - 1
// write the first product as out0[P0, r], the rest the second transposed as
// out1[r, P1].
__global__ __launch_bounds__(kThreads) void k_tn_reduce_pair(const float* __restrict__ part0, int splits0, int64_t P0,
                                                             float scale0, float* __restrict__ out0, int nb0,
                                                             const float* __restrict__ part1, int splits1, int64_t P1,
                                                             float scale1, float* __restrict__ out1, int r) {
  if ((int)blockIdx.x < nb0) tn_reduce_span(part0, splits0, P0, r, scale0, out0, blockIdx.x, nb0);
  else tn_reduce_t_block(part1, splits1, P1, r, scale1, out1, (int)blockIdx.x - nb0);
}

int grid_for(int64_t items) {
  int64_t g = (items + kThreads - 1) / kThreads;
  return (int)(g < 1 ? 1 : (g > 4096 ? 4096 : g));
}

// ---------------------------------------------------------------------------
// T = X L1 at decode-sized M (<= 16): fp32 partial sums over S slices of the
// reduction, part[s][m][c], each slice covering all r columns so that every
// 128-byte row of L1 is read by one work group.  Work group (b, s): columns
// 16 b .. 16 b + 15 of slice s, sixteen waves, one per virtual wave of
// tpart::slice_tile (32-row steps, one 16x16x32 MFMA each, the waves' results
// added in LDS in a fixed order).  The slices are summed in order s = 0 .. S-1
// by whoever needs T (the reduce kernel below, or the decode kernel), so every
// path gets the same T; the decode kernel can also form the slices itself with
// the same function.
// Stacked linears: G adapters L1_g [K, r] at L1 + g K r, all in one launch (the
// column tiles of segment g follow those of g - 1), slices of segment g at
// part + g S M r.
__global__ __launch_bounds__(64 * tpart::kVirt) void k_lora_part(const uint16_t* __restrict__ X, int64_t M, int64_t K,
                                                                const uint16_t* __restrict__ L1, int r, int64_t rows,
                                                                float* __restrict__ part) {
  __shared__ f32x4 red[tpart::kVirt * 64];
  const int ctiles = (r + 15) / 16;
  const int seg = blockIdx.x / ctiles;                    // stacked adapter of this work group
  tpart::slice_tile<tpart::kVirt>(X, M, K, L1 + (int64_t)seg * K * r, r, rows,
                                  part + (int64_t)seg * gridDim.y * M * r, (int)blockIdx.x - seg * ctiles,
                                  (int)blockIdx.y, red);
}

}  // namespace

int decode_t_slices(int64_t K) {
  const int64_t s = K / 512;
  return (int)(s < 1 ? 1 : (s > kDecodeTSlices ? kDecodeTSlices : s));
}

int64_t decode_t_rows(int64_t K) {
  const int S = decode_t_slices(K);
  return ((K + S - 1) / S + 31) / 32 * 32;
}

bool decode_t_ok(int64_t M, int64_t K, const void* X, const void* L1) {
  return M >= 1 && M <= 16 && (K % 64) == 0 && ((uintptr_t)X & 15) == 0 && ((uintptr_t)L1 & 1) == 0;
}

hipError_t launch_lora_part(const uint16_t* X, int64_t M, int64_t K, const uint16_t* L1, int r, float* part,
                            hipStream_t s, int G) {
  const int S = decode_t_slices(K);
  const int64_t rows = decode_t_rows(K);
  dim3 grid((unsigned)(G * ((r + 15) / 16)), (unsigned)S);
  hipLaunchKernelGGL(k_lora_part, grid, dim3(64 * tpart::kVirt), 0, s, X, M, K, L1, r, rows, part);
  return hipGetLastError();
}

// Split of a reduction of length R over `tiles` output tiles: about 768 work
// groups in all, but at most one slice per 512 of reduction, so that the fp32
// partials stay small next to the activation pass.
SplitPlan plan_rowsplit(int64_t tiles, int64_t R) {
  int64_t splits = (768 + tiles - 1) / tiles;
  const int64_t max_splits = R / 512;
  if (splits > max_splits) splits = max_splits;
  if (splits < 1) splits = 1;
  int64_t chunk = (R + splits - 1) / splits;
  chunk = (chunk + kTile - 1) / kTile * kTile;
  splits = (R + chunk - 1) / chunk;
  return SplitPlan{(int)splits, chunk};
}

// Split for the streaming kernel: about one work group per CU (64-row tiles
// times slices), each slice at least four 64-column steps long.
static SplitPlan plan_stream(int64_t tiles, int64_t R) {
  static const int cus = [] {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) !=
                                                hipSuccess || n < 1)
      n = 256;
    return n;
  }();
  int64_t splits = (cus + tiles / 2) / tiles;
  const int64_t max_splits = R / 256;
  if (splits > max_splits) splits = max_splits;
  if (splits < 1) splits = 1;
  int64_t chunk = (R + splits - 1) / splits;
  chunk = (chunk + kTile - 1) / kTile * kTile;
  splits = (R + chunk - 1) / chunk;
  return SplitPlan{(int)splits, chunk};
}

static bool skinny_stream_ok(const uint16_t* A, int64_t M, int64_t R, int64_t lda, const uint16_t* B, int r) {
  return (R % 8) == 0 && (lda % 8) == 0 && (r % 8) == 0 && r >= 8 && r <= 64 && ((uintptr_t)A & 15) == 0 &&
         ((uintptr_t)B & 15) == 0 && M * lda * 2 < (int64_t(1) << 31) && R * r * 2 < (int64_t(1) << 31);
}

// L2 [r, R] that buffer offsets do not reach: read by 64-bit address.
static bool past_2_31(int r, int64_t R) { return R * r * 2 >= (int64_t(1) << 31); }

size_t lora_skinny_ws(int64_t M, int64_t R, int r) {
  const int64_t tiles = (M + kTile - 1) / kTile;
  int64_t splits = std::max<int64_t>(plan_rowsplit(tiles, R).splits, plan_stream(tiles, R).splits);
  if (M <= 16) splits = std::max<int64_t>(splits, decode_t_slices(R));
  return (size_t)splits * M * r * sizeof(float);
}

hipError_t launch_lora_skinny(const uint16_t* A, int64_t M, int64_t R, int64_t lda, const uint16_t* B, bool b_is_kr,
                              int r, float scale, uint16_t* out, float* ws, hipStream_t s) {
  if (b_is_kr && lda == R && decode_t_ok(M, R, A, B)) {
    // decode-sized T: the slices the decode kernel also sums, added here in the same order
    hipError_t e = launch_lora_part(A, M, R, B, r, ws, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_skinny_reduce, dim3(grid_for((M * r + 3) / 4)), dim3(kThreads), 0, s, ws, decode_t_slices(R),
                       M * (int64_t)r, scale, out);
    return hipGetLastError();
  }
  const int64_t tiles = (M + kTile - 1) / kTile;
  if (skinny_stream_ok(A, M, R, lda, B, r)) {
    const SplitPlan sp = plan_stream(tiles, R);
    dim3 grid((unsigned)tiles, (unsigned)sp.splits);
    if (b_is_kr)
      hipLaunchKernelGGL((k_lora_skinny_stream<true>), grid, dim3(kSkThreads), 0, s, A, M, R, lda, B, r, sp.chunk, ws,
                         drop::Params{}, PackTo{});
    else
      hipLaunchKernelGGL((k_lora_skinny_stream<false>), grid, dim3(kSkThreads), 0, s, A, M, R, lda, B, r, sp.chunk, ws,
                         drop::Params{}, PackTo{});
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_skinny_reduce, dim3(grid_for((M * r + 3) / 4)), dim3(kThreads), 0, s, ws, sp.splits,
                       M * (int64_t)r, scale, out);
    return hipGetLastError();
  }
  const SplitPlan sp = plan_rowsplit(tiles, R);
  dim3 grid((unsigned)tiles, (unsigned)sp.splits);
  const bool avec = (R % 8) == 0 && (lda % 8) == 0 && ((uintptr_t)A & 15) == 0;
  const bool bvec = (b_is_kr ? (r % 8) == 0 : (R % 8) == 0) && ((uintptr_t)B & 15) == 0;
#define QL_SKINNY(BKR, VA, VB)                                                                                \
  hipLaunchKernelGGL((k_lora_skinny<BKR, VA, VB>), grid, dim3(kThreads), 0, s, A, M, R, lda, B, r, sp.chunk, ws, \
                     drop::Params{})
  if (b_is_kr) {
    if (R < 8) QL_SKINNY(true, kElements, kElements);
    else if (avec && bvec) QL_SKINNY(true, kPieces, kPieces);
    else if (avec && r < 8) QL_SKINNY(true, kPieces, kShort);
    else if (avec) QL_SKINNY(true, kPieces, kAnywhere);
    else if (bvec) QL_SKINNY(true, kAnywhere, kPieces);
    else if (r < 8) QL_SKINNY(true, kAnywhere, kShort);
    else QL_SKINNY(true, kAnywhere, kAnywhere);
  } else {
    if (past_2_31(r, R)) QL_SKINNY(false, kAnywhere, kFar);
    else if (R < 8) QL_SKINNY(false, kElements, kElements);
    else if (avec && bvec) QL_SKINNY(false, kPieces, kPieces);
    else if (avec) QL_SKINNY(false, kPieces, kAnywhere);
    else if (bvec) QL_SKINNY(false, kAnywhere, kPieces);
    else QL_SKINNY(false, kAnywhere, kAnywhere);
  }
#undef QL_SKINNY
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_skinny_reduce, dim3(grid_for((M * r + 3) / 4)), dim3(kThreads), 0, s, ws, sp.splits, M * (int64_t)r,
                     scale, out);
  return hipGetLastError();
}

size_t lora_tn_ws(int64_t M, int64_t P, int r) {
  const SplitPlan sp = plan_rowsplit((P + kTile - 1) / kTile, M);
  return (size_t)sp.splits * P * r * sizeof(float);
}

size_t lora_tn_pair_ws(int64_t M, int64_t P0, int64_t P1, int r) {
  return (lora_tn_ws(M, P0, r) + 255) / 256 * 256 + lora_tn_ws(M, P1, r);
}

hipError_t launch_lora_tn_pair(const uint16_t* A0, int64_t lda0, const uint16_t* B0, int64_t P0, float scale0,
                               float* out0, const uint16_t* A1, int64_t lda1, const uint16_t* B1, int64_t P1,
                               float scale1, float* out1_t, int64_t M, int r, float* ws, hipStream_t s) {
  const bool vec = (P0 % 8) == 0 && (lda0 % 8) == 0 && ((uintptr_t)A0 & 15) == 0 && (P1 % 8) == 0 &&
                   (lda1 % 8) == 0 && ((uintptr_t)A1 & 15) == 0 && (r % 8) == 0 && ((uintptr_t)B0 & 15) == 0 &&
                   ((uintptr_t)B1 & 15) == 0;
  float* part1 = ws + (lora_tn_ws(M, P0, r) + 255) / 256 * 256 / sizeof(float);
  if (!vec) {
    hipError_t e = launch_lora_tn(A0, lda0, B0, M, P0, r, scale0, false, out0, ws, s);
    if (e != hipSuccess) return e;
    return launch_lora_tn(A1, lda1, B1, M, P1, r, scale1, true, out1_t, part1, s);
  }
  const SplitPlan sp0 = plan_rowsplit((P0 + kTile - 1) / kTile, M);
  const SplitPlan sp1 = plan_rowsplit((P1 + kTile - 1) / kTile, M);
  const TnJob j0{A0, lda0, B0, P0, sp0.chunk, ws, (int)((P0 + kTile - 1) / kTile), sp0.splits};
  const TnJob j1{A1, lda1, B1, P1, sp1.chunk, part1, (int)((P1 + kTile - 1) / kTile), sp1.splits};
  const unsigned nwg = (unsigned)(j0.tiles * j0.splits + j1.tiles * j1.splits);
  hipLaunchKernelGGL((k_lora_tn_pair<kPieces, kPieces>), dim3(nwg), dim3(kThreads), 0, s, j0, j1, M, r);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int nb0 = grid_for((P0 * r + 3) / 4);
  const unsigned nb1 = (unsigned)((P1 + kTrP - 1) / kTrP);
  hipLaunchKernelGGL(k_tn_reduce_pair, dim3((unsigned)nb0 + nb1), dim3(kThreads), 0, s, ws, sp0.splits, P0, scale0,
                     out0, nb0, part1, sp1.splits, P1, scale1, out1_t, r);
  return hipGetLastError();
}

hipError_t launch_lora_tn(const uint16_t* A, int64_t lda, const uint16_t* B, int64_t M, int64_t P, int r,
                          float scale, bool transpose_out, float* out, float* ws, hipStream_t s) {
  const int64_t tiles = (P + kTile - 1) / kTile;
  const SplitPlan sp = plan_rowsplit(tiles, M);
  dim3 grid((unsigned)tiles, (unsigned)sp.splits);
  const bool avec = (P % 8) == 0 && (lda % 8) == 0 && ((uintptr_t)A & 15) == 0;
  const bool bvec = (r % 8) == 0 && ((uintptr_t)B & 15) == 0;
#define QL_TN(VA, VB) \
  hipLaunchKernelGGL((k_lora_tn<VA, VB>), grid, dim3(kThreads), 0, s, A, lda, B, M, P, r, sp.chunk, ws)
  if (P < 8 || M * r < 8) QL_TN(kElements, kElements);
  else if (avec && bvec) QL_TN(kPieces, kPieces);
  else if (avec && r < 8) QL_TN(kPieces, kShort);
  else if (avec) QL_TN(kPieces, kAnywhere);
  else if (bvec) QL_TN(kAnywhere, kPieces);
  else if (r < 8) QL_TN(kAnywhere, kShort);
  else QL_TN(kAnywhere, kAnywhere);
#undef QL_TN
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (transpose_out)
    hipLaunchKernelGGL(k_tn_reduce_t, dim3((unsigned)((P + kTrP - 1) / kTrP)), dim3(kThreads), 0, s, ws, sp.splits, P,
                       r, scale, out);
  else
    hipLaunchKernelGGL(k_tn_reduce, dim3(grid_for((P * r + 3) / 4)), dim3(kThreads), 0, s, ws, sp.splits, P, r, scale,
                       out);
  return hipGetLastError();
}

hipError_t launch_skinny_reduce(const float* part, int slices, int64_t n, float scale, uint16_t* out, hipStream_t s) {
  hipLaunchKernelGGL(k_skinny_reduce, dim3(grid_for((n + 3) / 4)), dim3(kThreads), 0, s, part, slices, n, scale, out);
  return hipGetLastError();
}

hipError_t launch_skinny_reduce3(const float* part, int slices, int64_t M, int r, float scale, const GPlanes& g,
                                 hipStream_t s) {
  const int rp = g_pitch(r);
  hipLaunchKernelGGL(k_skinny_reduce3, dim3(grid_for(M * rp / 4)), dim3(kThreads), 0, s, part, slices, M, r, rp, scale,
                     g.planes, rp == r ? nullptr : g.dense);
  return hipGetLastError();
}

// ---- with dropout, and with G kept to 24 bits ---------------------------------
// One pass over A [M, R] (dense): fp32 slices of the skinny product with B, of D o A with
// d.cut != 0 (L1 only), and A packed into `to` when that is given.
static hipError_t low_pass(const uint16_t* A, int64_t M, int64_t R, const uint16_t* B, bool b_is_kr, int r,
                           const drop::Params& d, uint8_t* codes, uint8_t* scales, float* ws, int* slices,
                           hipStream_t s) {
  const int64_t tiles = (M + kTile - 1) / kTile;
  if (skinny_stream_ok(A, M, R, R, B, r)) {
    const SplitPlan sp = plan_stream(tiles, R);
    const PackTo to{(uint32_t*)codes, scales, mx4::padded(R)};
    *slices = sp.splits;
    const dim3 grid((unsigned)tiles, (unsigned)sp.splits);
#define QL_LOW(BKR, D, Q)                                                                                           \
  hipLaunchKernelGGL((k_lora_skinny_stream<BKR, D, Q>), grid, dim3(kSkThreads), 0, s, A, M, R, R, B, r, sp.chunk, ws, \
                     d, to)
    if (!b_is_kr) {
      if (codes) QL_LOW(false, false, true);
      else QL_LOW(false, false, false);
    } else if (d.cut) {
      if (codes) QL_LOW(true, true, true);
      else QL_LOW(true, true, false);
    } else {
      if (codes) QL_LOW(true, false, true);
      else QL_LOW(true, false, false);
    }
#undef QL_LOW
    return hipGetLastError();
  }
  if (codes) {
    const hipError_t e = launch_mx4_quant(A, true, M, R, R, codes, scales, s);
    if (e != hipSuccess) return e;
  }
  const SplitPlan sp = plan_rowsplit(tiles, R);
  *slices = sp.splits;
  const dim3 grid((unsigned)tiles, (unsigned)sp.splits);
  const bool vec = (R % 8) == 0;
#define QL_LOW(BKR, VA, VB, D)                                                                                     \
  hipLaunchKernelGGL((k_lora_skinny<BKR, VA, VB, D>), grid, dim3(kThreads), 0, s, A, M, R, R, B, r, sp.chunk, ws, d)
  if (!b_is_kr) {
    if (past_2_31(r, R)) QL_LOW(false, kAnywhere, kFar, false);
    else if (vec) QL_LOW(false, kPieces, kPieces, false);
    else if (R < 8) QL_LOW(false, kElements, kElements, false);
    else QL_LOW(false, kAnywhere, kAnywhere, false);
  } else if (d.cut) {
    if (R < 8) QL_LOW(true, kElements, kElements, true);
    else if (r < 8 && vec) QL_LOW(true, kPieces, kShort, true);
    else if (r < 8) QL_LOW(true, kAnywhere, kShort, true);
    else if (vec) QL_LOW(true, kPieces, kAnywhere, true);
    else QL_LOW(true, kAnywhere, kAnywhere, true);
  } else {
    if (R < 8) QL_LOW(true, kElements, kElements, false);
    else if (r < 8 && vec) QL_LOW(true, kPieces, kShort, false);
    else if (r < 8) QL_LOW(true, kAnywhere, kShort, false);
    else if (vec) QL_LOW(true, kPieces, kAnywhere, false);
    else QL_LOW(true, kAnywhere, kAnywhere, false);
  }
#undef QL_LOW
  return hipGetLastError();
}

hipError_t launch_lora_down_drop(const uint16_t* X, int64_t M, int64_t K, const uint16_t* L1, int r,
                                 const drop::Params& d, uint16_t* T, uint8_t* codes, uint8_t* scales, float* ws,
                                 hipStream_t s) {
  if (d.cut == 0 && !codes) return launch_lora_skinny(X, M, K, K, L1, true, r, 1.0f, T, ws, s);
  int slices = 0;
  const hipError_t e = low_pass(X, M, K, L1, true, r, d, codes, scales, ws, &slices, s);
  if (e != hipSuccess) return e;
  return launch_skinny_reduce(ws, slices, M * r, d.cut ? d.scale : 1.0f, T, s);
}

hipError_t launch_lora_grad_in3(const uint16_t* dY, int64_t M, int64_t N, const uint16_t* L2, int r, float scale,
                                const GPlanes& G, uint8_t* codes, uint8_t* scales, float* ws, hipStream_t s) {
  int slices = 0;
  const hipError_t e = low_pass(dY, M, N, L2, false, r, drop::Params{}, codes, scales, ws, &slices, s);
  if (e != hipSuccess) return e;
  return launch_skinny_reduce3(ws, slices, M, r, scale, G, s);
}

hipError_t launch_lora_slices(const uint16_t* A, int64_t M, int64_t R, const uint16_t* B, bool b_is_kr, int r, float* ws,
                              int* slices, hipStream_t s) {
  return low_pass(A, M, R, B, b_is_kr, r, drop::Params{}, nullptr, nullptr, ws, slices, s);
}

hipError_t launch_lora_grads3(const uint16_t* X, int64_t K, const uint16_t* G, const drop::Params& d, float* dL1,
                              const uint16_t* dY, int64_t N, const uint16_t* T, float scale, float* dL2, int64_t M,
                              int r, float* ws, hipStream_t s) {
  if (lora_grads_wide_ok(M, K, N, r))
    return launch_lora_grads_wide(X, K, G, d, dL1, dY, N, T, scale, dL2, M, r, ws, s);
  const bool vec = (K % 8) == 0 && (N % 8) == 0, vect = (r % 8) == 0;
  float* part1 = ws + (lora_tn_ws(M, K, r) + 255) / 256 * 256 / sizeof(float);
  const SplitPlan sp0 = plan_rowsplit((K + kTile - 1) / kTile, M);
  const SplitPlan sp1 = plan_rowsplit((N + kTile - 1) / kTile, M);
  const bool whole = sp0.splits == 1 && sp1.splits == 1;
  const TnJob j0{X, K, G, K, sp0.chunk, whole ? dL1 : ws, (int)((K + kTile - 1) / kTile), sp0.splits};
  const TnJob j1{dY, N, T, N, sp1.chunk, whole ? dL2 : part1, (int)((N + kTile - 1) / kTile), sp1.splits};
  const float s0 = whole ? d.scale : 1.0f, s1 = whole ? scale : 1.0f;
  const unsigned nwg = (unsigned)(j0.tiles * j0.splits + j1.tiles * j1.splits);
#define QL_TN3(V, T)                                                                                                \
  do {                                                                                                              \
    if (d.cut)                                                                                                      \
      hipLaunchKernelGGL((k_lora_tn_pair3<V, T, true>), dim3(nwg), dim3(kThreads), 0, s, j0, j1, M, r, g_pitch(r), d, \
                         s0, s1, whole);                                                                            \
    else                                                                                                            \
      hipLaunchKernelGGL((k_lora_tn_pair3<V, T, false>), dim3(nwg), dim3(kThreads), 0, s, j0, j1, M, r, g_pitch(r), d, \
                         s0, s1, whole);                                                                            \
  } while (0)
  if (K < 8 || N < 8 || M * r < 8) QL_TN3(kElements, kElements);
  else if (vec && vect) QL_TN3(kPieces, kPieces);
  else if (vec && r < 8) QL_TN3(kPieces, kShort);
  else if (vec) QL_TN3(kPieces, kAnywhere);
  else if (r < 8) QL_TN3(kAnywhere, kShort);
  else if (vect) QL_TN3(kAnywhere, kPieces);
  else QL_TN3(kAnywhere, kAnywhere);
#undef QL_TN3
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || whole) return e;
  return launch_tn_reduce_pair(ws, sp0.splits, K, d.scale, dL1, part1, sp1.splits, N, scale, dL2, r, s);
}

hipError_t launch_tn_reduce_pair(const float* part0, int splits0, int64_t P0, float scale0, float* out0,
                                 const float* part1, int splits1, int64_t P1, float scale1, float* out1_t, int r,
                                 hipStream_t s) {
  const int nb0 = grid_for((P0 * r + 3) / 4);
  const unsigned nb1 = (unsigned)((P1 + kTrP - 1) / kTrP);
  hipLaunchKernelGGL(k_tn_reduce_pair, dim3((unsigned)nb0 + nb1), dim3(kThreads), 0, s, part0, splits0, P0, scale0, out0,
                     nb0, part1, splits1, P1, scale1, out1_t, r);
  return hipGetLastError();
}

size_t lora_grads3_ws(int64_t M, int64_t K, int64_t N, int r) {
  return lora_grads_wide_ok(M, K, N, r) ? lora_grads_wide_ws(M, K, N, r) : lora_tn_pair_ws(M, K, N, r);
}
