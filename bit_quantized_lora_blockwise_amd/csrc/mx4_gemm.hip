// Products of two microscaled 4-bit matrices (layout: mx4.h) on the scaled matrix
// instruction, with the adapter term in the same tile:
//   C[m][p] = bf16(sum_b 2^(ea + eb) sum_{32} a b + adapter[m][p]),  A [M, R], B [P, R]
//   forward   adapter = s (T L2)         T [M, r], L2 [r, P]
//   backward  adapter = D o (G L1^T)     G [M, r], L1 [P, r]
// fp32 accumulators throughout, one rounding at the end.
#include <type_traits>

#include "mx4.h"

#include "kernels.h"

namespace {

using namespace mx4;

constexpr int kStages = 4;        // reduction steps of 128 in LDS
constexpr int kPL = 64 + 8;       // pitch of [row][c] adapter tiles
constexpr uint32_t kOOB = 0x80000000u;   // past every buffer: loads read 0, stores are dropped

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}

// Loads to LDS (16 or 4 bytes a lane, lane l's at dst + 16 l or 4 l).  Issued from
// inline assembly, which writes no register, so that the compiler makes no LDS
// read wait for them; the kernels' own waits count them.  M0 holds the LDS address
// and is put back, since the compiler does not track it across assembly.
__device__ __forceinline__ void dma16(uint32_t dst, uint32_t vo, __amdgpu_buffer_rsrc_t rs, uint32_t so) {
  uint32_t keep;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
      : "=&s"(keep)
      : "s"(__builtin_amdgcn_readfirstlane(dst)), "v"(vo), "s"(rs), "s"(__builtin_amdgcn_readfirstlane(so))
      : "memory");
}
__device__ __forceinline__ void dma4(uint32_t dst, uint32_t vo, __amdgpu_buffer_rsrc_t rs, uint32_t so) {
  uint32_t keep;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dword %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
      : "=&s"(keep)
      : "s"(__builtin_amdgcn_readfirstlane(dst)), "v"(vo), "s"(rs), "s"(__builtin_amdgcn_readfirstlane(so))
      : "memory");
}

// Origin (in tiles) of virtual work group v: XCD x (v % 8 = x) takes a contiguous run of
// the nt tiles, ordered in bands of eight tile rows, down each band's columns: the
// 32 tiles an XCD holds at a time then share 8 + 4 tiles' operands in its L2.
__device__ __forceinline__ void tile_at(int v, int tm, int tp, int nt, int& im, int& ip) {
  const int per = nt / 8, extra = nt % 8, xcd = v % 8, q = v / 8;
  const int tile = xcd < extra ? xcd * (per + 1) + q : extra * (per + 1) + (xcd - extra) * per + q;
  const int band = tile / (8 * tp), rows = min(8, tm - 8 * band), in = tile - band * 8 * tp;
  im = __builtin_amdgcn_readfirstlane(8 * band + in % rows);
  ip = __builtin_amdgcn_readfirstlane(in / rows);
}

// One 32 x 32 accumulator tile of C: lane half h holds columns 8 g + 4 h + e,
// e = 0..3, of its row; a swap of the halves of a register pair gives half h
// columns 16 gp + 8 h .. +7, one 16-byte store.  vo: the lane's byte offset in C of
// its row and of column 8 h of the wave's first tile (out of range for a row past
// the end: the hardware drops the store); off: columns from there to this tile;
// left: columns of C from column 8 h of this tile on.
// kPieces: in whole 16-byte pieces, at any address (P % 8 == 0, or the tile is inside).
template <bool kPieces>
__device__ __forceinline__ void store_tile(const f32x16& v, __amdgpu_buffer_rsrc_t rc, uint32_t vo, int off, int left) {
#pragma unroll
  for (int gp = 0; gp < 2; ++gp) {
    const u32x2 x = __builtin_amdgcn_permlane32_swap(qk::pack_bf16x2(v[8 * gp], v[8 * gp + 1]),
                                                     qk::pack_bf16x2(v[8 * gp + 4], v[8 * gp + 5]), false, false);
    const u32x2 y = __builtin_amdgcn_permlane32_swap(qk::pack_bf16x2(v[8 * gp + 2], v[8 * gp + 3]),
                                                     qk::pack_bf16x2(v[8 * gp + 6], v[8 * gp + 7]), false, false);
    const u32x4 o = {x[0], y[0], x[1], y[1]};
    const int at = 2 * (off + 16 * gp), n = left - 16 * gp;
    if constexpr (kPieces) {
      __builtin_amdgcn_raw_buffer_store_b128(o, rc, n > 0 ? vo + at : kOOB, 0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(o[e >> 1] >> (16 * (e & 1))), rc,
                                              e < n ? vo + at + 2 * e : kOOB, 0, 0);
    }
  }
}

// All of a wave's tiles: rows m, m + 32, ... (m this lane's) and columns p0, p0 + 32, ...
template <bool kPieces, int kMT, int kPT>
__device__ __forceinline__ void store_tiles(const f32x16 (&acc)[kMT][kPT], uint16_t* __restrict__ C, int m, int p0, int M,
                                            int P) {
  const __amdgpu_buffer_rsrc_t rc = rsrc(C, (uint64_t)M * P * 2);
  int h = (threadIdx.x & 63) >> 5;
  asm volatile("" : "+v"(h));               // addresses are formed here, not held through the reduction
#pragma unroll
  for (int i = 0; i < kMT; ++i) {
    const uint32_t vo = m + 32 * i < M ? 2u * ((uint32_t)(m + 32 * i) * (uint32_t)P + p0 + 8 * h) : kOOB;
#pragma unroll
    for (int j = 0; j < kPT; ++j) store_tile<kPieces>(acc[i][j], rc, vo, 32 * j, P - p0 - 8 * h - 32 * j);
  }
}

// Rows of no whole 16-byte pieces: waves whose columns end inside the matrix store whole
// pieces all the same, those on the edge single elements (which throughout took 130 us
// of a 4093 x 11007 product).
template <int kMT, int kPT>
__device__ __forceinline__ void store_any(const f32x16 (&acc)[kMT][kPT], uint16_t* __restrict__ C, int m, int p0, int M,
                                          int P) {
  if (p0 + 32 * kPT <= P) store_tiles<true, kMT, kPT>(acc, C, m, p0, M, P);
  else store_tiles<false, kMT, kPT>(acc, C, m, p0, M, P);
}

// kMode: 0 no adapter, 1 forward, 2 backward, 3 backward with dropout.
// Tile kWM x kWP waves of (32 kMT) x (32 kPT), one scale chunk a wave.
template <int kMode, int kWM, int kWP, int kMT, int kPT>
struct Gemm {
  static constexpr int kWaves = kWM * kWP, kThreads = 64 * kWaves;
  static constexpr int kBM = 32 * kMT * kWM, kBP = 32 * kPT * kWP;
  static constexpr int kCodesA = kBM * 64, kCodesB = kBP * 64;          // bytes of a step
  static constexpr int kStage = kCodesA + kCodesB + 4 * (kBM + kBP);
  static constexpr int kChunksA = kBM / 16, kChunksB = kBP / 16;        // of 64 rows of one block position (1 KB)
  static constexpr int kPerA = kChunksA / kWaves, kPerB = kChunksB / kWaves;
  static constexpr int kPerS = (kBM + kBP) / 64 / kWaves;               // 64 rows' scale words each
  static_assert(kChunksA % kWaves == 0 && kChunksB % kWaves == 0 && (kBM + kBP) / 64 % kWaves == 0,
                "loads spread evenly");
  static constexpr int kLoads = kPerA + kPerB + kPerS;                  // of a wave and step
  // adapter operands, over stages 2 and 3 and what follows them
  static constexpr int kPD = kBP + 8;                                   // pitch of the forward's [c][p] tile
  static constexpr int kLA = kBM * kPL * 2, kLB = kMode == 1 ? 64 * kPD * 2 : kBP * kPL * 2;
  static constexpr int kBits = kMode == 3 ? kBM * drop::bit_pitch(kBP) : 0;
  static constexpr int kAdapter = kMode == 0 ? 0 : kLA + kLB + kBits;
  static constexpr int kLds = 2 * kStage + (kAdapter > 2 * kStage ? kAdapter : 2 * kStage);
  static_assert(kLds <= 160 * 1024, "fits the LDS of a CU");
};

// Smaller products: 128 x 128 tiles, four waves of 64 x 64, two work groups a CU, four LDS
// stages.  The adapter's product comes first, while the first stages load, and starts the
// sums.  Bound: filling and draining the pipeline and, with few tiles, the latency of a step
// (0.45 us with one work group a CU): 1024 x 4096 -> 8192 24 us (2.9 PFLOP/s), 256 x 11008 ->
// 4096 a whole forward 35 us.
template <int kMode, int kWM, int kWP, int kMT, int kPT>
__global__ __launch_bounds__(64 * kWM * kWP) void k_mx4_gemm(const uint8_t* __restrict__ ac,
                                                             const uint8_t* __restrict__ as, int M,
                                                             const uint8_t* __restrict__ bc,
                                                             const uint8_t* __restrict__ bs, int P, int words,
                                                             Mx4Lora lo, uint16_t* __restrict__ C) {
  using G = Gemm<kMode, kWM, kWP, kMT, kPT>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[G::kLds];
  const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63;
  const int wm = w % kWM, wp = w / kWM, h = l >> 5;

  const int tm = (M + G::kBM - 1) / G::kBM, tp = (P + G::kBP - 1) / G::kBP;
  int m0, p0;
  tile_at(blockIdx.x, tm, tp, tm * tp, m0, p0);
  m0 *= G::kBM;
  p0 *= G::kBP;

  // ---- loads to LDS.  A stage holds codes A [4][kBM][16], codes B [4][kBP][16],
  // scales A [kBM][4], scales B [kBP][4].  Rows past the end repeat the last one:
  // their results are not stored.
  const __amdgpu_buffer_rsrc_t rac = rsrc(ac, (uint64_t)words * 64 * M), rbc = rsrc(bc, (uint64_t)words * 64 * P);
  uint32_t va[G::kPerA], vb[G::kPerB], vs[G::kPerS];
#pragma unroll
  for (int i = 0; i < G::kPerA; ++i) va[i] = 16u * min(m0 + 64 * ((w + i * G::kWaves) % (G::kBM / 64)) + l, M - 1);
#pragma unroll
  for (int i = 0; i < G::kPerB; ++i) vb[i] = 16u * min(p0 + 64 * ((w + i * G::kWaves) % (G::kBP / 64)) + l, P - 1);
#pragma unroll
  for (int i = 0; i < G::kPerS; ++i) {
    const int c = w + i * G::kWaves, cb = c - G::kBM / 64;
    vs[i] = 4u * (cb < 0 ? min(m0 + 64 * c + l, M - 1) : min(p0 + 64 * cb + l, P - 1));
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS_AS uint8_t*)lds;
  // Load n (of kLoads) of step q into its stage.
  auto load = [&](int q, int n) {
    const uint32_t st = lds0 + (uint32_t)(q % kStages) * G::kStage;
    if (n < G::kPerA) {
      const int c = w + n * G::kWaves;                       // chunk: block position c / (kBM / 64)
      dma16(st + 1024u * c, va[n], rac, (uint32_t)(4 * q + c / (G::kBM / 64)) * 16u * (uint32_t)M);
    } else if (n < G::kPerA + G::kPerB) {
      const int c = w + (n - G::kPerA) * G::kWaves;
      dma16(st + G::kCodesA + 1024u * c, vb[n - G::kPerA], rbc, (uint32_t)(4 * q + c / (G::kBP / 64)) * 16u * (uint32_t)P);
    } else {
      const int i = n - G::kPerA - G::kPerB, c = w + i * G::kWaves;
      const bool of_a = c < G::kBM / 64;
      const uint32_t rows = of_a ? M : P;
      dma4(st + G::kCodesA + G::kCodesB + 256u * c, vs[i], rsrc(of_a ? as : bs, (uint64_t)words * 4 * rows),
           (uint32_t)q * 4u * rows);
    }
  };
  auto issue = [&](int q) {
#pragma unroll
    for (int n = 0; n < G::kLoads; ++n) load(q, n);
  };

  // ---- fragments of half s of a step: lane half h takes block 2 h + s of its row,
  // whose scale is byte s of the 16 bits at 2 h of the row's scale word.
  // Read n (of kMT + kPT): a row's codes; the first half's bring its scale as well.
  struct Frags {
    u32x4 a[kMT], b[kPT];
  };
  struct Scales {
    uint32_t a[kMT], b[kPT];
  };
  const LDS_AS uint8_t* const smem = (const LDS_AS uint8_t*)lds;
  const int ra = 32 * kMT * wm + (l & 31), rb = 32 * kPT * wp + (l & 31);
  auto read = [&](int q, int s, int n, Frags& f, Scales& sc) {
    const LDS_AS uint8_t* st = smem + (q % kStages) * G::kStage;
    const LDS_AS uint8_t* ss = st + G::kCodesA + G::kCodesB + 2 * h;
    if (n < kMT) {
      f.a[n] = *(const LDS_AS u32x4*)(st + ((2 * h + s) * G::kBM + ra + 32 * n) * 16);
      if (s == 0) sc.a[n] = *(const LDS_AS uint16_t*)(ss + 4 * (ra + 32 * n));
    } else {
      f.b[n - kMT] = *(const LDS_AS u32x4*)(st + G::kCodesA + ((2 * h + s) * G::kBP + rb + 32 * (n - kMT)) * 16);
      if (s == 0) sc.b[n - kMT] = *(const LDS_AS uint16_t*)(ss + 4 * (G::kBM + rb + 32 * (n - kMT)));
    }
  };
  // The rows of an accumulator are columns of C (operand order B, A): a lane holds
  // four neighbouring columns of one row of C.
  f32x16 acc[kMT][kPT];
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kPT; ++j) acc[i][j] = f32x16{};

  issue(0);
  if (words > 1) issue(1);

  // ---- adapter term
  if constexpr (kMode != 0) {
    LDS_AS uint16_t* const la = (LDS_AS uint16_t*)((LDS_AS uint8_t*)lds + 2 * G::kStage);
    LDS_AS uint16_t* const lb = la + G::kLA / 2;
    LDS_AS uint8_t* const bits = (LDS_AS uint8_t*)(lb + G::kLB / 2);
    const int r = lo.r;
    for (int i = t; i < G::kBM * 8; i += G::kThreads) {
      const int row = i >> 3, c = (i & 7) * 8;
      u32x4 v = {0, 0, 0, 0};
      if (m0 + row < M && c < r) v = qk::load8_row(lo.A + (int64_t)(m0 + row) * r, c, r);
      *(LDS_AS u32x4*)(la + row * kPL + c) = v;
    }
    if constexpr (kMode == 1) {
      for (int i = t; i < 64 * (G::kBP / 8); i += G::kThreads) {
        const int c = i / (G::kBP / 8), p = (i % (G::kBP / 8)) * 8;
        u32x4 v = {0, 0, 0, 0};
        if (c < r && p0 + p < P) v = qk::load8_row(lo.B + (int64_t)c * P, p0 + p, P);
        *(LDS_AS u32x4*)(lb + c * G::kPD + p) = v;
      }
    } else {
      for (int i = t; i < G::kBP * 8; i += G::kThreads) {
        const int row = i >> 3, c = (i & 7) * 8;
        u32x4 v = {0, 0, 0, 0};
        if (p0 + row < P && c < r) v = qk::load8_row(lo.B + (int64_t)(p0 + row) * r, c, r);
        *(LDS_AS u32x4*)(lb + row * kPL + c) = v;
      }
    }
    if constexpr (kMode == 3) drop::fill_bits<G::kBM, G::kBP>(bits, lo.d, m0, p0, t, G::kThreads);
    __syncthreads();
    for (int s = 0; s < (r + 15) / 16; ++s) {
      bf16x8 a[kMT], b[kPT];
#pragma unroll
      for (int i = 0; i < kMT; ++i) a[i] = qk::frag_rowmajor(la, kPL, 32 * (kMT * wm + i), 16 * s);
#pragma unroll
      for (int j = 0; j < kPT; ++j)
        b[j] = kMode == 1 ? qk::frag_kmajor(lb, G::kPD, 16 * s, 32 * (kPT * wp + j))
                          : qk::frag_rowmajor(lb, kPL, 32 * (kPT * wp + j), 16 * s);
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kPT; ++j) acc[i][j] = qk::mfma32(b[j], a[i], acc[i][j]);
    }
    if constexpr (kMode == 1) {
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kPT; ++j) acc[i][j] *= lo.scale;
    }
    if constexpr (kMode == 3) {
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kPT; ++j) {
          // the 32 decisions of this lane's row of the 32 x 32 tile
          const uint32_t b = *(const LDS_AS uint32_t*)(bits + (ra + 32 * i) * drop::bit_pitch(G::kBP) + 4 * (kPT * wp + j)) >>
                             (4 * h);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            acc[i][j][e] = (b >> (8 * (e >> 2) + (e & 3))) & 1u ? lo.d.scale * acc[i][j][e] : 0.0f;
        }
    }
    __syncthreads();
  }

  // ---- reduction.  Step q's second half is read while its first half multiplies;
  // then one barrier (stage q is read by every wave, stage q + 1 has arrived) lets
  // step q + 4 go into stage q's buffer and the first half of q + 1 be read
  // while the second half multiplies: the matrix unit has work on both sides of
  // the barrier.
  if (words > 2) issue(2);
  if (words > 3) issue(3);
  auto wait = [&](int ahead) {          // all but the loads of the last `ahead` steps have arrived
    if (ahead >= 3) asm volatile("s_waitcnt vmcnt(%0)" ::"i"(3 * G::kLoads) : "memory");
    else if (ahead == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"i"(2 * G::kLoads) : "memory");
    else if (ahead == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"i"(G::kLoads) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  };
  auto barrier = [&]() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
  Frags f0, f1;
  Scales sc, sn;
  constexpr int kMfma = kMT * kPT, kReads = kMT + kPT;
  wait(min(words - 1, 3));
  barrier();
#pragma unroll
  for (int n = 0; n < kReads; ++n) read(0, 0, n, f0, sc);
  // One step with kLeft steps after it (4: four or more).  Between two products a
  // wave issues one read or load: they go out in the shadow of the matrix unit.
  auto step = [&](int q, auto left_c) __attribute__((always_inline)) {
    constexpr int kLeft = decltype(left_c)::value;
#pragma unroll
    for (int n = 0; n < kMfma; ++n) {
      const int i = n % kMT, j = n / kMT;
      acc[i][j] = mx4::mfma32<0, 0>(f0.b[j], sc.b[j], f0.a[i], sc.a[i], acc[i][j]);
      if (n < kReads) read(q, 1, n, f1, sc);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int n = kMfma; n < kReads; ++n) read(q, 1, n, f1, sc);
    if constexpr (kLeft > 0) {
      wait(kLeft >= 3 ? 2 : kLeft - 1);
      barrier();
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < kMfma; ++n) {
      const int i = n % kMT, j = n / kMT;
      acc[i][j] = mx4::mfma32<1, 1>(f1.b[j], sc.b[j], f1.a[i], sc.a[i], acc[i][j]);
      if (kLeft > 0 && n < kReads) read(q + 1, 0, n, f0, sn);
      if (kLeft > 3 && n < G::kLoads) load(q + 4, n);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kLeft > 0) {
#pragma unroll
      for (int n = kMfma; n < kReads; ++n) read(q + 1, 0, n, f0, sn);
      sc = sn;
    }
    if constexpr (kLeft > 3) {
#pragma unroll
      for (int n = kMfma; n < G::kLoads; ++n) load(q + 4, n);
    }
  };
  int q = 0;
  for (; q + 4 < words; ++q) step(q, std::integral_constant<int, 4>{});
  if (words - q == 4) step(q++, std::integral_constant<int, 3>{});
  if (words - q == 3) step(q++, std::integral_constant<int, 2>{});
  if (words - q == 2) step(q++, std::integral_constant<int, 1>{});
  step(q, std::integral_constant<int, 0>{});

  if ((P & 7) == 0) store_tiles<true, kMT, kPT>(acc, C, m0 + ra, p0 + 32 * kPT * wp, M, P);
  else store_any<kMT, kPT>(acc, C, m0 + ra, p0 + 32 * kPT * wp, M, P);
}

// ---------------------------------------------------------------------------
// Large products: 256 x 256 tiles on a persistent grid, eight waves of 64 x 128
// (two a SIMD, 128 accumulators a lane).  One ring of four LDS stages of 34 KB runs
// through all tiles of a work group: after a tile's last reduction step come its
// two adapter operands as stages of their own, then the next tile's steps, so that
// the matrix unit finds the next tile's operands in LDS when a tile ends.  The
// adapter product comes last, one 32 x 32 tile of it at a time on top of the base
// sums, between them and the store.  The dropout decisions of the tile are drawn
// during the reduction, a Philox round between two products: the vector unit is
// free while the other wave's product runs, where a draw before the loop took 8 us
// a tile.
// Bound: the matrix unit under the chip's power limit.  A step of 128 of one round of 256
// tiles takes 0.82 to 0.88 us on random data (5.2 to 4.9 PFLOP/s; 0.48 to 0.52 us on zeros,
// and 6.7 PFLOP/s is what the products alone reach on random data); the clock is then about
// 1.85 GHz and the matrix unit busy half of its cycles (2048 x 8192 x 22016 with the adapter:
// 189 to 206 us, on zeros 139 to 144, the last of 2.7 rounds of tiles and 10 us of launch,
// first loads and last stores among them; no LDS bank conflicts).  4096 x 11008 x 4096 backward with dropout 115 us.  A P that is no multiple
// of 8 costs in the stores: 4093 x 4097 -> 11007 157 us, -> 11008 120 us.
constexpr int kRT = 512;                    // threads
constexpr int kRB = 256;                    // tile edge
constexpr int kRCodes = kRB * 64;           // bytes of one operand's codes in a step
constexpr int kRStage = 2 * kRCodes + 8 * kRB;
constexpr int kRLoads = 5;                  // of a wave and step: 4 of codes, 1 of scale words
constexpr int kRMinWords = 6;               // reduction steps that the ring needs

// Adapter operand stages.  [row][c], 128 bytes a row: 16-byte piece c of row i in
// slot c ^ (i / 2 % 8).  [c][p], 512 bytes a row: piece p of row c in slot p ^ 4 (c % 4).
// With these, the 32 lanes of a (transposed) fragment read meet no bank twice.
__device__ __forceinline__ int slot_rc(int row, int c) { return row * 128 + 16 * (c ^ ((row >> 1) & 7)); }
__device__ __forceinline__ int slot_cp(int c, int p) { return c * 512 + 16 * (p ^ (4 * (c & 3))); }

// kVec: P % 8 == 0 and, with an adapter, r % 8 == 0: 16-byte pieces everywhere.
template <int kMode, bool kVec>
__global__ __launch_bounds__(kRT, 2) void k_mx4_gemm_ring(const uint8_t* __restrict__ ac,
                                                          const uint8_t* __restrict__ as, int M,
                                                          const uint8_t* __restrict__ bc,
                                                          const uint8_t* __restrict__ bs, int P, int words, Mx4Lora lo,
                                                          uint16_t* __restrict__ C) {
  constexpr int kMT = 2, kPT = 4;
  constexpr bool kDrop = kMode == 3;
  constexpr int kDraws = kRB * kRB / 8 / kRT;       // Philox calls of a thread and tile
  __shared__ __attribute__((aligned(16))) uint8_t lds[kStages * kRStage + (kDrop ? kRB * drop::bit_pitch(kRB) : 0)];
  const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63;
  const int wm = w & 3, wp = w >> 2, h = l >> 5;
  const LDS_AS uint8_t* const smem = (const LDS_AS uint8_t*)lds;
  LDS_AS uint8_t* const bits = (LDS_AS uint8_t*)lds + kStages * kRStage;
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

  const int tm = (M + kRB - 1) / kRB, tp = (P + kRB - 1) / kRB, nt = tm * tp;
  auto place = [&](int v, int& m0, int& p0) {
    tile_at(v, tm, tp, nt, m0, p0);
    m0 *= kRB;
    p0 *= kRB;
  };

  // ---- loads (as above: rows past the end repeat the last one)
  const __amdgpu_buffer_rsrc_t rac = rsrc(ac, (uint64_t)words * 64 * M), rbc = rsrc(bc, (uint64_t)words * 64 * P);
  const bool scale_a = w < 4;
  const uint32_t srows = scale_a ? M : P;
  const __amdgpu_buffer_rsrc_t rsc = rsrc(scale_a ? as : bs, (uint64_t)words * 4 * srows);
  struct Rows {
    uint32_t a, b, s;        // lane offsets: 64 rows of A, of B, of the scale words
  };
  // Wave w's loads n = 0, 1 (A) and 2, 3 (B) bring block positions w / 4 + 2 (n % 2),
  // rows 64 (w % 4) .. +63.
  auto rows_of = [&](int m0, int p0) {
    Rows r;
    r.a = 16u * min(m0 + 64 * (w & 3) + l, M - 1);
    r.b = 16u * min(p0 + 64 * (w & 3) + l, P - 1);
    r.s = 4u * (scale_a ? min(m0 + 64 * w + l, M - 1) : min(p0 + 64 * (w - 4) + l, P - 1));
    return r;
  };
  auto load = [&](const Rows& r, int q, int ring, int n) {
    const uint32_t st = lds0 + (uint32_t)(ring & (kStages - 1)) * kRStage;
    const int kb = (w >> 2) + 2 * (n & 1);
    const uint32_t dst = st + 4096u * kb + 1024u * (w & 3);
    if (n < 2) dma16(dst, r.a, rac, (uint32_t)(4 * q + kb) * 16u * (uint32_t)M);
    else if (n < 4) dma16(dst + kRCodes, r.b, rbc, (uint32_t)(4 * q + kb) * 16u * (uint32_t)P);
    else dma4(st + 2 * kRCodes + 256u * w, r.s, rsc, (uint32_t)q * 4u * srows);
  };

  // ---- adapter operands: 32 KB each, four loads a wave.  Rows whose 16-byte pieces
  // are whole and aligned go straight to LDS (pieces past the matrix read as zeros);
  // others are sent as zeros and written over by hand before they are read.
  const int r = kMode ? lo.r : 0;
  const __amdgpu_buffer_rsrc_t rla = rsrc(lo.A, (uint64_t)M * r * 2), rlb = rsrc(lo.B, (uint64_t)P * r * 2);
  auto load_rc = [&](__amdgpu_buffer_rsrc_t rs, int row0, int rows, int ring, int n) {
    const int row = 32 * w + 8 * n + (l >> 3), c = (l & 7) ^ ((row >> 1) & 7);
    const bool ok = kVec && row0 + row < rows && 8 * c < r;
    dma16(lds0 + (uint32_t)(ring & (kStages - 1)) * kRStage + 4096u * w + 1024u * n,
          ok ? (uint32_t)((row0 + row) * r + 8 * c) * 2u : kOOB, rs, 0);
  };
  auto load_cp = [&](int p0, int ring, int n) {
    const int c = 8 * w + 2 * n + (l >> 5), p = 8 * ((l & 31) ^ (4 * (c & 3)));
    const bool ok = kVec && c < r && p0 + p < P;
    dma16(lds0 + (uint32_t)(ring & (kStages - 1)) * kRStage + 4096u * w + 1024u * n,
          ok ? (uint32_t)(c * P + p0 + p) * 2u : kOOB, rlb, 0);
  };

  struct Frags {
    u32x4 a[kMT], b[kPT];
  };
  struct Scales {
    uint32_t a[kMT], b[kPT];
  };
  const int ra = 64 * wm + (l & 31), rb = 128 * wp + (l & 31);
  auto read = [&](int ring, int s, int n, Frags& f, Scales& sc) {
    const LDS_AS uint8_t* st = smem + (ring & (kStages - 1)) * kRStage;
    const LDS_AS uint8_t* ss = st + 2 * kRCodes + 2 * h;
    if (n < kMT) {
      f.a[n] = *(const LDS_AS u32x4*)(st + ((2 * h + s) * kRB + ra + 32 * n) * 16);
      if (s == 0) sc.a[n] = *(const LDS_AS uint16_t*)(ss + 4 * (ra + 32 * n));
    } else {
      f.b[n - kMT] = *(const LDS_AS u32x4*)(st + kRCodes + ((2 * h + s) * kRB + rb + 32 * (n - kMT)) * 16);
      if (s == 0) sc.b[n - kMT] = *(const LDS_AS uint16_t*)(ss + 4 * (kRB + rb + 32 * (n - kMT)));
    }
  };
  auto barrier = [&]() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

  int m0, p0, v = blockIdx.x;
  place(v, m0, p0);
  Rows cur = rows_of(m0, p0);
#pragma unroll
  for (int q = 0; q < kStages; ++q)
#pragma unroll
    for (int n = 0; n < kRLoads; ++n) load(cur, q, q, n);
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(2 * kRLoads) : "memory");
  barrier();

  // On top of each tile: steps 0 and 1 are in LDS for every wave, 2 and 3 on their way.
  int ring0 = 0;
  for (;;) {
    const int vn = v + (int)gridDim.x;
    const bool more = vn < nt;
    int m1, p1;
    place(more ? vn : v, m1, p1);            // with no next tile this one's first steps are fetched again, unread
    const Rows next = rows_of(m1, p1);
    f32x16 acc[kMT][kPT];
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
      for (int j = 0; j < kPT; ++j) acc[i][j] = f32x16{};

    Frags f0, f1;
    Scales sc, sn;
    drop::State ph;
    int drawn = 0;
    auto draw_begin = [&]() {
      const int f = drawn * kRT + t;
      ph = drop::begin(lo.d, (uint32_t)(m0 + (f >> 5)), (uint32_t)(p0 >> 3) + (f & 31));
    };
    auto draw_end = [&]() {
      const int f = drawn * kRT + t;
      bits[(f >> 5) * drop::bit_pitch(kRB) + (f & 31)] = (uint8_t)drop::bits8_of(u32x4{ph.c0, ph.c1, ph.c2, ph.c3}, lo.d.cut);
      ++drawn;
    };
    // Step q with kLeft steps after it (4: four or more); kFirst: its successor needs no wait.
    auto step = [&](int q, auto left_c, auto first_c, auto draw_c) __attribute__((always_inline)) {
      constexpr int kLeft = decltype(left_c)::value;
      constexpr bool kFirst = decltype(first_c)::value, kDraw = decltype(draw_c)::value;
      const int ring = ring0 + q;
      if constexpr (kDraw) draw_begin();
#pragma unroll
      for (int n = 0; n < kMT * kPT; ++n) {
        const int i = n % kMT, j = n / kMT;
        acc[i][j] = mx4::mfma32<0, 0>(f0.b[j], sc.b[j], f0.a[i], sc.a[i], acc[i][j]);
        if (n < kMT + kPT) read(ring, 1, n, f1, sc);
        if constexpr (kDraw) {
          if (n & 1) drop::round(ph);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // steps 2 and 3 on their way, and of the adapter's loads and the next tile's what was issued after step q + 1
      constexpr int kNewer = kLeft >= 3 ? 2 * kRLoads : kMode == 0 ? 2 * kRLoads : kLeft == 2 ? kRLoads + 4 : 8;
      if constexpr (!kFirst && kLeft > 0) asm volatile("s_waitcnt vmcnt(%0)" ::"i"(kNewer) : "memory");
      barrier();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n < kMT * kPT; ++n) {
        const int i = n % kMT, j = n / kMT;
        acc[i][j] = mx4::mfma32<1, 1>(f1.b[j], sc.b[j], f1.a[i], sc.a[i], acc[i][j]);
        if (kLeft > 0 && n < kMT + kPT) read(ring + 1, 0, n, f0, sn);
        // into this step's buffer: step q + 4, or after the last step the adapter's operands and the next tile's steps
        if constexpr (kLeft > 3) {
          if (n < kRLoads) load(cur, q + 4, ring + 4, n);
        } else if constexpr (kMode == 0) {
          if (n < kRLoads) load(next, 3 - kLeft, ring + 4, n);
        } else if constexpr (kLeft == 3) {
          if (n < 4) load_rc(rla, m0, M, ring + 4, n);
        } else if constexpr (kLeft == 2) {
          if (n < 4) {
            if constexpr (kMode == 1) load_cp(p0, ring + 4, n);
            else load_rc(rlb, p0, P, ring + 4, n);
          }
        } else {
          if (n < kRLoads) load(next, 1 - kLeft, ring + 4, n);
        }
        if constexpr (kDraw) {
          if ((n & 1) && n < 7) drop::round(ph);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (kDraw) draw_end();
      if constexpr (kLeft > 0) sc = sn;
    };
    using std::false_type;
    using std::true_type;
    using Four = std::integral_constant<int, 4>;
#pragma unroll
    for (int n = 0; n < kMT + kPT; ++n) read(ring0, 0, n, f0, sc);
    step(0, Four{}, true_type{}, std::integral_constant<bool, kDrop>{});
    int q = 1;
    if constexpr (kDrop)
      for (; q + 4 < words && drawn < kDraws; ++q) step(q, Four{}, false_type{}, true_type{});
    for (; q + 4 < words; ++q) step(q, Four{}, false_type{}, false_type{});
    step(q, std::integral_constant<int, 3>{}, false_type{}, false_type{});
    step(q + 1, std::integral_constant<int, 2>{}, false_type{}, false_type{});
    step(q + 2, std::integral_constant<int, 1>{}, false_type{}, false_type{});
    step(q + 3, std::integral_constant<int, 0>{}, false_type{}, false_type{});

    if constexpr (kMode == 0) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"i"(2 * kRLoads) : "memory");     // the next tile's steps 0 and 1
      barrier();
    } else {
      LDS_AS uint8_t* const la = (LDS_AS uint8_t*)lds + ((ring0 + words) & (kStages - 1)) * kRStage;
      LDS_AS uint8_t* const lb = (LDS_AS uint8_t*)lds + ((ring0 + words + 1) & (kStages - 1)) * kRStage;
      // the products stay above what follows: without this the compiler sinks the last
      // steps' past the loops below, with all their operands held
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kPT; ++j) asm volatile("" : "+v"(acc[i][j]));
      if constexpr (kDrop)
#pragma clang loop vectorize(disable) unroll(disable)
        while (drawn < kDraws) {
          draw_begin();
#pragma unroll
          for (int n = 0; n < 7; ++n) drop::round(ph);
          draw_end();
        }
      asm volatile("s_waitcnt vmcnt(%0)" ::"i"(2 * kRLoads) : "memory");
      barrier();
      if constexpr (!kVec) {
        for (int i = t; i < kRB * 8; i += kRT) {
          const int row = i >> 3, c = i & 7;
          u32x4 x = {0, 0, 0, 0};
          if (m0 + row < M && 8 * c < r) x = qk::load8_row(lo.A + (int64_t)(m0 + row) * r, 8 * c, r);
          *(LDS_AS u32x4*)(la + slot_rc(row, c)) = x;
          x = u32x4{0, 0, 0, 0};
          if constexpr (kMode == 1) {
            const int cc = i >> 5, p = i & 31;
            if (cc < r && p0 + 8 * p < P) x = qk::load8_row(lo.B + (int64_t)cc * P, p0 + 8 * p, P);
            *(LDS_AS u32x4*)(lb + slot_cp(cc, p)) = x;
          } else {
            if (p0 + row < P && 8 * c < r) x = qk::load8_row(lo.B + (int64_t)(p0 + row) * r, 8 * c, r);
            *(LDS_AS u32x4*)(lb + slot_rc(row, c)) = x;
          }
        }
        barrier();
      }
      // a row's piece 2 s + h and, [c][p], a transposed read (each 16 lanes a 4 x 16
      // block): only the piece's slot depends on the lane, rows go into the offset
      int lx = l;
      asm volatile("" : "+v"(lx));          // as in store_tiles
      const int hx = lx >> 5, swz = (lx >> 1) & 7;
      auto frag_rc = [&](const LDS_AS uint8_t* base, int row0, int s) {
        return *(const LDS_AS bf16x8*)(base + (lx & 31) * 128 + 16 * ((2 * s + hx) ^ swz) + row0 * 128);
      };
      const int g = lx >> 4, i4 = lx & 15;
      const int tr0 = (((g >> 1) << 3) + (i4 >> 2)) * 512 + 16 * (2 * (g & 1) + ((i4 & 3) >> 1)) + 8 * (i4 & 1);
      auto frag_cp = [&](const LDS_AS uint8_t* base, int j, int s) {
        const LDS_AS uint8_t* at = base + tr0 + 16 * (4 * j ^ 4 * (i4 >> 2)) + s * 16 * 512 + wp * 256;
        const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4*)at);
        const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4*)(at + 4 * 512));
        const u32x2 a = __builtin_bit_cast(u32x2, x), b = __builtin_bit_cast(u32x2, y);
        return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
      };
      // the operands are zero past r; a barrier for the scheduler after each 32 x 32
      // tile keeps it from holding several tiles' products in registers
#pragma unroll
      for (int j = 0; j < kPT; ++j) {
        bf16x8 fb[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) fb[s] = kMode == 1 ? frag_cp(lb, j, s) : frag_rc(lb, 128 * wp + 32 * j, s);
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
          f32x16 x = {};
#pragma unroll
          for (int s = 0; s < 4; ++s) x = qk::mfma32(fb[s], frag_rc(la, 64 * wm + 32 * i, s), x);
          if constexpr (kMode == 1) acc[i][j] += lo.scale * x;
          if constexpr (kMode == 2) acc[i][j] += x;
          if constexpr (kDrop) {
            // the 32 decisions of this lane's row of the 32 x 32 tile
            const uint32_t keep =
                *(const LDS_AS uint32_t*)(bits + (ra + 32 * i) * drop::bit_pitch(kRB) + 4 * (kPT * wp + j)) >> (4 * h);
#pragma unroll
            for (int e = 0; e < 16; ++e) {   // the bit spread over a word clears what is dropped
              const uint32_t m = (uint32_t)__builtin_amdgcn_sbfe((int)keep, 8 * (e >> 2) + (e & 3), 1);
              acc[i][j][e] += lo.d.scale * __uint_as_float(__float_as_uint(x[e]) & m);
            }
          }
          asm volatile("" ::: "memory");
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // the next tile's steps 0 and 1
      barrier();                                             // and every wave is past the adapter's buffers
    }
    if constexpr (kVec) store_tiles<true, kMT, kPT>(acc, C, m0 + ra, p0 + 128 * wp, M, P);
    else store_any<kMT, kPT>(acc, C, m0 + ra, p0 + 128 * wp, M, P);
    if (!more) break;
    ring0 += words;
    if constexpr (kMode != 0) {
      ring0 += 2;
#pragma unroll
      for (int q2 = 2; q2 < 4; ++q2)
#pragma unroll
        for (int n = 0; n < kRLoads; ++n) load(next, q2, ring0 + q2, n);
    }
    v = vn;
    m0 = m1;
    p0 = p1;
    cur = next;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");           // no load to LDS outlives the work group
}

template <int kMode, bool kVec>
hipError_t launch_ring(const uint8_t* ac, const uint8_t* as, int64_t M, const uint8_t* bc, const uint8_t* bs, int64_t P,
                       int64_t R, const Mx4Lora& lora, uint16_t* C, hipStream_t s) {
  const int64_t tiles = (M + kRB - 1) / kRB * ((P + kRB - 1) / kRB);
  static const int cus = [] {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 8)
      n = 256;
    return n / 8 * 8;
  }();
  hipLaunchKernelGGL((k_mx4_gemm_ring<kMode, kVec>), dim3((unsigned)(tiles < cus ? tiles : cus)), dim3(kRT), 0, s, ac, as, (int)M,
                     bc, bs, (int)P, (int)(padded(R) / kPad), lora, C);
  return hipGetLastError();
}

template <int kMode, int kWM, int kWP, int kMT, int kPT>
hipError_t launch(const uint8_t* ac, const uint8_t* as, int64_t M, const uint8_t* bc, const uint8_t* bs, int64_t P,
                  int64_t R, const Mx4Lora& lora, uint16_t* C, hipStream_t s) {
  using G = Gemm<kMode, kWM, kWP, kMT, kPT>;
  const int64_t tiles = (M + G::kBM - 1) / G::kBM * ((P + G::kBP - 1) / G::kBP);
  hipLaunchKernelGGL((k_mx4_gemm<kMode, kWM, kWP, kMT, kPT>), dim3((unsigned)tiles), dim3(G::kThreads), 0, s, ac, as,
                     (int)M, bc, bs, (int)P, (int)(padded(R) / kPad), lora, C);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_gemm(const uint8_t* ac, const uint8_t* as, int64_t M, const uint8_t* bc, const uint8_t* bs,
                           int64_t P, int64_t R, const Mx4Lora& lora, uint16_t* C, hipStream_t s) {
  // The smaller tiles run two to a CU: while all of them fit on the chip at once they win,
  // then the ring does.  Small and ring, us: 512 tiles of 128 x 128 (1024 x 4096 -> 8192) 24
  // and 30, whole forward 42 and 45, backward 66 and 70; 516 (768 x 4096 -> 11008) 32 and 30,
  // 54 and 45, 78 and 70; 256 (1024 x 4096 -> 4096) 16 and 26.
  const bool big = ((M + 127) / 128) * ((P + 127) / 128) > 512 && padded(R) / kPad >= kRMinWords;
  const bool vec = P % 8 == 0 && (!lora.A || lora.r % 8 == 0);
#define QL_MX(MODE)                                                                                      \
  return !big ? launch<MODE, 2, 2, 2, 2>(ac, as, M, bc, bs, P, R, lora, C, s)                            \
              : (vec ? launch_ring<MODE, true> : launch_ring<MODE, false>)(ac, as, M, bc, bs, P, R, lora, C, s)
  if (!lora.A) QL_MX(0);
  if (!lora.bwd) QL_MX(1);
  if (lora.d.cut == 0) QL_MX(2);
  QL_MX(3);
#undef QL_MX
}
