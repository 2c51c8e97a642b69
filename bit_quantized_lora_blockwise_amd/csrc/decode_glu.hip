// The gated product for up to 16 rows (decoding): H = bf16(silu(G) U), [G | U] = X W'^T + s T L2
// for a stacked gate|up weight W [2 F, K] in NF4, in one pass over its codes.
//
// Work group: 16 columns of H, eight waves: four take the 16 gate rows, four the 16 up rows,
// and split the reduction in steps of 256 columns.  In a step, lane (g = l / 16, x = l % 16)
// holds block g of row x (64 weights, 32 bytes of codes), rebuilds it eight weights at a time
// (dequant.h) and multiplies it against X on the 16x16x32 instruction, the next step's
// codes in flight.  At most 80 registers, so that three work groups share a CU.  X is staged
// in LDS in the order that the lookups give the weights in; it, T's slices and L2 are
// requested before the codes.  The waves' sums meet in LDS in order, where the gate meets its up
// half, so neither goes to memory.
//
// One row 4096 -> 2 x 11008: 17.4 us, 47 MB at 2.7 TB/s (9 us at a copy's rate); 8192 -> 2 x 22016 55 us.
// Bound: the vector units, 4.15 instructions a weight, busy for 90% of the time that a CU has work;
// the rest is the first loads' latency and the last work groups (2.7 a CU).  T's slices take 2.4 us
// in a launch before it: formed in this one, behind flags as for a single linear, the two together
// took as long (19.2 us), and the wait's fallback cost registers.
#include "dequant.h"
#include "glu.h"
#include "kernels.h"

namespace {

using namespace nf4;

constexpr int kWv = 8, kHalf = 4, kThr = 64 * kWv;
constexpr int kXBytes = 32768;
constexpr int kSlices = 8;
constexpr uint32_t kOOB = 0x80000000u;

typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}

struct Step {
  u32x4 cw[2];
  uint8_t c2b;                     // kept a byte: its widening is not scheduled at the load
  float c1v;
};

// kXPer: 16-byte pieces of X a thread stages.  kVecR: r % 4 == 0.
template <int kXPer, bool kVecR>
__global__ __launch_bounds__(kThr, 6) void k_glu_decode(const uint16_t* __restrict__ X, int M, int K, int F,
                                                        const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ c2, const float* __restrict__ c1,
                                                        const float* __restrict__ Tp, int S, uint16_t* __restrict__ T_out,
                                                        const uint16_t* __restrict__ L2, int r, float scale,
                                                        uint16_t* __restrict__ H, Nf4Params p) {
  __shared__ __attribute__((aligned(16))) uint8_t xl[kXBytes + 128];   // 128 bytes of zeros behind X, for rows past M
  __shared__ f32x4 red[kWv][64];
  const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, g = l >> 4, x = l & 15;
  const int half = w >> 2, wh = w & 3;
  const int n = 16 * (int)blockIdx.x + x;
  const uint32_t kb = (uint32_t)K / 64, kb_lim = n < F ? kb : 0u;
  const uint64_t N = 2 * (uint64_t)F;
  const SplitConst kc = split_const();
  const __amdgpu_buffer_rsrc_t rc = rsrc(codes, N * (K / 2)), r2 = rsrc(c2, N * kb),
                               r1 = rsrc(c1, 4 * ((N * kb + 255) / 256)), rx = rsrc(X, (uint64_t)M * K * 2);
  uint32_t blk_row = ((uint32_t)(half ? F : 0) + n) * kb;
  asm volatile("" : "+v"(blk_row));        // formed before the loads whose registers its product may borrow

  u32x4 xr[kXPer];
  const uint32_t xbytes = (uint32_t)M * K * 2;
#pragma unroll
  for (int j = 0; j < kXPer; ++j) {
    const uint32_t o = 16u * (uint32_t)(t + j * kThr);
    xr[j] = __builtin_amdgcn_raw_buffer_load_b128(rx, o < xbytes ? o : kOOB, 0, 0);
  }
  // the adapter's operands of this wave's 16 ranks: lane (g, x) ranks rb .. + 3 of T's row x and of L2's column n
  const int rb = 16 * wh + 4 * g;
  const bool t_ok = rb < r && x < M;
  f32x4 ps[kSlices];
  {
    const __amdgpu_buffer_rsrc_t rp = rsrc(Tp + (int64_t)half * S * M * r, 4 * (uint64_t)S * M * r);
    const uint32_t at = 4 * (uint32_t)(x * r + rb);
#pragma unroll
    for (int s = 0; s < kSlices; ++s) {
      const uint32_t o = t_ok && s < S ? at + (uint32_t)(4 * s * M * r) : kOOB;
      if constexpr (kVecR) {
        ps[s] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rp, o, 0, 0));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ps[s][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rp, rb + j < r ? o + 4 * j : kOOB, 0, 0));
      }
    }
  }
  uint16_t vl[4];
  {
    const uint16_t* l2 = L2 + (int64_t)half * r * F;
#pragma unroll
    for (int j = 0; j < 4; ++j) vl[j] = rb + j < r && n < F ? l2[(int64_t)(rb + j) * F + n] : 0;
  }
  __builtin_amdgcn_sched_barrier(0);
  auto load = [&](uint32_t s, Step& st) {  // step s of this wave: blocks 4 (wh + 4 s) + g; zeros past its last
    const uint32_t b = 4 * ((uint32_t)wh + kHalf * s) + g;
    const bool ok = b < kb_lim;
    const uint32_t co = ok ? 32u * (blk_row + b) : kOOB;
    st.cw[0] = __builtin_amdgcn_raw_buffer_load_b128(rc, co, 0, 0);
    st.cw[1] = __builtin_amdgcn_raw_buffer_load_b128(rc, co + 16, 0, 0);
    st.c2b = __builtin_amdgcn_raw_buffer_load_b8(r2, ok ? blk_row + b : kOOB, 0, 0);
    st.c1v = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r1, ok ? 4 * ((blk_row + b) >> 8) : kOOB, 0, 0));
  };
  Step sa, sb;
  load(0, sa);
  __builtin_amdgcn_sched_barrier(0);
  {
    f32x4 tv = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < kSlices; ++s)
      if (s < S) tv += ps[s];
    red[w][l] = tv;                        // this lane's own until the sums meet there
  }
#pragma unroll
  for (int j = 0; j < kXPer; ++j) {
    const uint32_t o = 16u * (uint32_t)(t + j * kThr);
    const u32x4 v = xr[j];                 // columns as (0, 2, 4, 6, 1, 3, 5, 7)
    const u32x4 e = {__builtin_amdgcn_perm(v[1], v[0], 0x05040100u), __builtin_amdgcn_perm(v[3], v[2], 0x05040100u),
                     __builtin_amdgcn_perm(v[1], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)};
    if (o < xbytes) *(LDS_AS u32x4*)((LDS_AS uint8_t*)xl + o) = e;
  }
  if (t < 8) *(LDS_AS u32x4*)((LDS_AS uint8_t*)xl + kXBytes + 16 * t) = u32x4{0, 0, 0, 0};
  __syncthreads();

  f32x4 acc = {0, 0, 0, 0};
  auto compute = [&](uint32_t s, const Step& st) {
    const BlockLut lut = make_lut(qk::e4m3fn_to_f32(st.c2b) * st.c1v, p);
    const uint32_t b = 4 * ((uint32_t)wh + kHalf * s) + g;
    const LDS_AS u32x4* xs = (const LDS_AS u32x4*)((const LDS_AS uint8_t*)xl +
                                                   (x < M && b < kb ? ((uint32_t)x * K + 64 * b) * 2u : (uint32_t)kXBytes));
#pragma unroll
    for (int d = 0; d < 8; ++d)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xs[d]),
                                                    __builtin_bit_cast(bf16x8, dequant8_eo(lut, st.cw[d >> 2][d & 3], kc)),
                                                    acc, 0, 0, 0);
  };
  const uint32_t nsteps = (kb + 3) / 4;
  const uint32_t nst = nsteps > (uint32_t)wh ? (nsteps - wh + kHalf - 1) / kHalf : 0u;   // uniform
  uint32_t i = 0;
  for (; i + 2 <= nst; i += 2) {
    load(i + 1, sb);
    __builtin_amdgcn_sched_barrier(0);
    compute(i, sa);
    load(i + 2, sa);
    __builtin_amdgcn_sched_barrier(0);
    compute(i + 1, sb);
  }
  if (i < nst) compute(i, sa);
  {
    uint16_t a0 = vl[0], a1 = vl[1], a2 = vl[2], a3 = vl[3];
    asm volatile("" : "+v"(a0), "+v"(a1), "+v"(a2), "+v"(a3));
    const u32x2 b = {__builtin_amdgcn_perm(a1, a0, 0x05040100u), __builtin_amdgcn_perm(a3, a2, 0x05040100u)};
    f32x4 low = {0, 0, 0, 0}, tv = red[w][l];
    // T in three planes, 24 bits, as every path of the gated product takes it
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const u32x2 a = {qk::pack_bf16x2(tv[0], tv[1]), qk::pack_bf16x2(tv[2], tv[3])};
      low = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, a), __builtin_bit_cast(s16x4, b), low, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (k == 0 && T_out && blockIdx.x == 0 && t_ok && rb + j < r)
          T_out[((int64_t)half * M + x) * r + rb + j] = (uint16_t)(a[j >> 1] >> (16 * (j & 1)));
        tv[j] -= __uint_as_float(j & 1 ? a[j >> 1] & 0xFFFF0000u : a[j >> 1] << 16);
      }
    }
    acc += scale * low;
  }
  red[w][l] = acc;
  __syncthreads();
  if (w == 0) {
    f32x4 gt = red[0][l], up = red[kHalf][l];
#pragma unroll
    for (int k = 1; k < kHalf; ++k) {
      gt += red[k][l];
      up += red[kHalf + k][l];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {          // lane: row 4 g + j, column n
      const int m = 4 * g + j;
      if (m < M && n < F) H[(int64_t)m * F + n] = qk::f32_to_bf16(glu::silu(gt[j]) * up[j]);
    }
  }
}

}  // namespace

bool glu_decode_ok(int64_t M, int64_t K) { return M <= 16 && M * K * 2 <= kXBytes; }

hipError_t launch_glu_decode(const uint16_t* X, int64_t M, int64_t K, int64_t F, const uint8_t* codes, const uint8_t* c2,
                             const float* c1, const float* Tp, int S, uint16_t* T_out, const uint16_t* L2, int r,
                             float scale, uint16_t* H, hipStream_t s) {
  const dim3 grid((unsigned)((F + 15) / 16));
#define QL_GD(N, V)                                                                                                 \
  hipLaunchKernelGGL((k_glu_decode<N, V>), grid, dim3(kThr), 0, s, X, (int)M, (int)K, (int)F, codes, c2, c1, Tp, S, \
                     T_out, L2, r, scale, H, nf4_params())
#define QL_GDR(N)                   \
  do {                              \
    if (r % 4 == 0) QL_GD(N, true); \
    else QL_GD(N, false);           \
  } while (0)
  if (M * K * 2 <= 16 * kThr) QL_GDR(1);
  else if (M * K * 2 <= 32 * kThr) QL_GDR(2);
  else QL_GDR(4);
#undef QL_GDR
#undef QL_GD
  return hipGetLastError();
}
