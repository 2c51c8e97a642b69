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

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}

// 8 consecutive bf16 of a row starting at column `col`, zero past `ncols`.
__device__ __forceinline__ u32x4 load_row8(const uint16_t* __restrict__ row, int64_t col, int64_t ncols) {
  const uint16_t* p = row + col;
  if (col + 8 <= ncols && ((uintptr_t)p & 15) == 0) return *(const u32x4*)p;
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t h = (col + j < ncols) ? p[j] : 0;
    v[j >> 1] |= h << (16 * (j & 1));
  }
  return v;
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
  static_assert(kChunksA % kWaves == 0 && kChunksB % kWaves == 0 && (kBM + kBP) / 64 == kWaves, "loads spread evenly");
  static constexpr int kLoads = kPerA + kPerB + 1;                      // of a wave and step
  // adapter operands, over stages 2 and 3 and what follows them
  static constexpr int kPD = kBP + 8;                                   // pitch of the forward's [c][p] tile
  static constexpr int kLA = kBM * kPL * 2, kLB = kMode == 1 ? 64 * kPD * 2 : kBP * kPL * 2;
  static constexpr int kBits = kMode == 3 ? kBM * drop::bit_pitch(kBP) : 0;
  static constexpr int kAdapter = kMode == 0 ? 0 : kLA + kLB + kBits;
  static constexpr int kLds = 2 * kStage + (kAdapter > 2 * kStage ? kAdapter : 2 * kStage);
  static_assert(kLds <= 160 * 1024, "fits the LDS of a CU");
};

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

  // ---- tile: XCD x (work groups x, x + 8, ...) takes a contiguous run of tiles,
  // ordered in bands of eight tile rows, down each band's columns: the 32 tiles an
  // XCD holds at a time then share 8 + 4 tiles' operands in its L2.
  const int tm = (M + G::kBM - 1) / G::kBM, tp = (P + G::kBP - 1) / G::kBP, nt = tm * tp;
  int m0, p0;
  {
    const int per = nt / 8, extra = nt % 8, xcd = blockIdx.x % 8, q = blockIdx.x / 8;
    const int tile = xcd < extra ? xcd * (per + 1) + q : extra * (per + 1) + (xcd - extra) * per + q;
    const int band = tile / (8 * tp), rows = min(8, tm - 8 * band), in = tile - band * 8 * tp;
    m0 = (8 * band + in % rows) * G::kBM;
    p0 = in / rows * G::kBP;
  }

  // ---- loads to LDS.  A stage holds codes A [4][kBM][16], codes B [4][kBP][16],
  // scales A [kBM][4], scales B [kBP][4].  Rows past the end repeat the last one:
  // their results are not stored.
  const __amdgpu_buffer_rsrc_t rac = rsrc(ac, (uint64_t)words * 64 * M), rbc = rsrc(bc, (uint64_t)words * 64 * P);
  const bool scale_a = w < G::kBM / 64;
  const int srows = scale_a ? M : P;
  const __amdgpu_buffer_rsrc_t rsc = rsrc(scale_a ? as : bs, (uint64_t)words * 4 * srows);
  uint32_t va[G::kPerA], vb[G::kPerB], vs;
#pragma unroll
  for (int i = 0; i < G::kPerA; ++i) va[i] = 16u * min(m0 + 64 * ((w + i * G::kWaves) % (G::kBM / 64)) + l, M - 1);
#pragma unroll
  for (int i = 0; i < G::kPerB; ++i) vb[i] = 16u * min(p0 + 64 * ((w + i * G::kWaves) % (G::kBP / 64)) + l, P - 1);
  vs = 4u * min((scale_a ? m0 : p0) + 64 * (scale_a ? w : w - G::kBM / 64) + l, srows - 1);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS_AS uint8_t*)lds;
  // Issued from inline assembly, which writes no register, so that the compiler
  // makes no LDS read wait for them; the waits before the barriers count them.
  // M0 holds the LDS address and is put back, since the compiler does not track
  // it across assembly.
  auto dma16 = [&](uint32_t dst, uint32_t vo, __amdgpu_buffer_rsrc_t rs, uint32_t so) {
    uint32_t keep;
    asm volatile(
        "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
        : "=&s"(keep)
        : "s"(__builtin_amdgcn_readfirstlane(dst)), "v"(vo), "s"(rs), "s"(__builtin_amdgcn_readfirstlane(so))
        : "memory");
  };
  auto dma4 = [&](uint32_t dst, uint32_t vo, __amdgpu_buffer_rsrc_t rs, uint32_t so) {
    uint32_t keep;
    asm volatile(
        "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dword %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
        : "=&s"(keep)
        : "s"(__builtin_amdgcn_readfirstlane(dst)), "v"(vo), "s"(rs), "s"(__builtin_amdgcn_readfirstlane(so))
        : "memory");
  };
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
      dma4(st + G::kCodesA + G::kCodesB + 256u * w, vs, rsc, (uint32_t)q * 4u * (uint32_t)srows);
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
      if (m0 + row < M && c < r) v = load_row8(lo.A + (int64_t)(m0 + row) * r, c, r);
      *(LDS_AS u32x4*)(la + row * kPL + c) = v;
    }
    if constexpr (kMode == 1) {
      for (int i = t; i < 64 * (G::kBP / 8); i += G::kThreads) {
        const int c = i / (G::kBP / 8), p = (i % (G::kBP / 8)) * 8;
        u32x4 v = {0, 0, 0, 0};
        if (c < r && p0 + p < P) v = load_row8(lo.B + (int64_t)c * P, p0 + p, P);
        *(LDS_AS u32x4*)(lb + c * G::kPD + p) = v;
      }
    } else {
      for (int i = t; i < G::kBP * 8; i += G::kThreads) {
        const int row = i >> 3, c = (i & 7) * 8;
        u32x4 v = {0, 0, 0, 0};
        if (p0 + row < P && c < r) v = load_row8(lo.B + (int64_t)(p0 + row) * r, c, r);
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

  // ---- store: lane (h, m) holds columns 8 g + 4 h + e, e = 0..3, of row m; a swap of
  // the halves of a register pair gives half h columns 16 gp + 8 h .. +7
#pragma unroll
  for (int i = 0; i < kMT; ++i) {
    const int m = m0 + ra + 32 * i;
#pragma unroll
    for (int j = 0; j < kPT; ++j)
#pragma unroll
      for (int gp = 0; gp < 2; ++gp) {
        const f32x16 v = acc[i][j];
        const u32x2 x = __builtin_amdgcn_permlane32_swap(qk::pack_bf16x2(v[8 * gp], v[8 * gp + 1]),
                                                         qk::pack_bf16x2(v[8 * gp + 4], v[8 * gp + 5]), false, false);
        const u32x2 y = __builtin_amdgcn_permlane32_swap(qk::pack_bf16x2(v[8 * gp + 2], v[8 * gp + 3]),
                                                         qk::pack_bf16x2(v[8 * gp + 6], v[8 * gp + 7]), false, false);
        const u32x4 o = {x[0], y[0], x[1], y[1]};
        const int p = p0 + 32 * (kPT * wp + j) + 16 * gp + 8 * h;
        if (m < M && p < P) {
          uint16_t* dst = C + (int64_t)m * P + p;
          if ((P & 7) == 0) {
            *(u32x4*)dst = o;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (p + e < P) dst[e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
          }
        }
      }
  }
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
  const bool big = ((M + 255) / 256) * ((P + 255) / 256) >= 128;
#define QL_MX(MODE)                                                              \
  return big ? launch<MODE, 4, 2, 2, 4>(ac, as, M, bc, bs, P, R, lora, C, s)     \
             : launch<MODE, 2, 2, 2, 2>(ac, as, M, bc, bs, P, R, lora, C, s)
  if (!lora.A) QL_MX(0);
  if (!lora.bwd) QL_MX(1);
  if (lora.d.cut == 0) QL_MX(2);
  QL_MX(3);
#undef QL_MX
}
