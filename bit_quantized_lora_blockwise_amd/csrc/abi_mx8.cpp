// Entry points of the 8-bit activations, of the norm and of the gated product: argument
// checks, workspace layout and dispatch.  Contracts: include/qlora.h.
#include <algorithm>
#include <cmath>

#include "abi_util.h"
#include "mx8.h"
#include "side_stream.h"

namespace {

using namespace qlabi;

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr drop::Params kNoDrop{0, 0, 0, 0, 0, 1.0f};

bool matrix_ok(int64_t rows, int64_t cols, int64_t ld) {
  return rows > 0 && cols > 0 && rows < kLim && cols < kLim && ld >= cols && ld <= kMaxElems / rows &&
         cols <= kMaxElems / rows - 32;
}

// Sizes of a layer over the NF4 base, as qlora_linear_fwd's: X and dX, Y and dY and W's codes
// each below 2^31 bytes, and each factor of the adapters; n is the number of W's rows and ldy that of
// Y's columns as the kernels keep it, halves that of the adapters.
bool layer_ok(int64_t M, int64_t K, int64_t n, int64_t ldy, int r, int halves = 1) {
  return M > 0 && K > 0 && n > 0 && K % 64 == 0 && r >= 1 && r <= 64 && M < kLim && K < kLim && n < kLim &&
         M * K < kLim / 2 && ldy < kLim && M * ldy < kLim / 2 && n * (K / 2) < kLim && n * r < kLim / 2 &&
         halves * K * r < kLim / 2;
}

bool glu_ok(int64_t M, int64_t K, int64_t F, int r) {
  return F > 0 && F < kLim / 2 && layer_ok(M, K, 2 * F, (2 * F + 7) / 8 * 8, r, 2);
}

// Whether T goes into the product as slices, which it adds up itself (a launch less): where the
// product is one of those for few rows, while the rank-r product has at most 128 tiles of 16 x 16
// (past 64 its launch takes one slice a tile).  Whole calls with 8-bit copies, us, planes of their
// own / slices: 1024 -> 2 x 2752 17 rows 37 / 31, 128 rows 40 / 31; 2048 -> 2 x 1000 500 rows (128
// tiles) 46 / 37, 1000 rows (252) 63 / 63; 8192 -> 2 x 256 1000 rows 67 / 76.
bool few_ok(int64_t M, int64_t K, int64_t F, int r) {
  return (M + 15) / 16 * ((r + 15) / 16) <= 128 && glu_small_ok(M, K, F);
}

// Forward: [T's planes of both halves][fp32 slices of both].
struct FwdWs {
  size_t planes, part, total;
};
FwdWs fwd_ws(int64_t M, int64_t K, int64_t F, int r) {
  FwdWs w{0, round_up(few_ok(M, K, F, r) ? mx4_small_ws(M, r) : lora_skinny_ws(M, K, r)), 0};
  if (!few_ok(M, K, F, r)) w.planes = round_up((size_t)6 * M * g_pitch(r) * 2);
  w.total = w.planes + 2 * w.part;
  return w;
}

// Whether dX [M, K], whose reduction walks n columns (both planes of dZ), is taken in slices of the reduction.  The work
// groups of the product for few rows (64 columns of 32 rows) and of the large tiles each walk all of
// it; slices cost a launch and the partial sums' way to memory.  Whole backwards, us, walked / in
// slices: gated, K = 4096, n = 22016 1 row 91 / 69, 64 rows 120 / 73, 512 rows 456 / 154, 1024 rows
// 505 / 246; K = 1024, n = 5504 64 rows 49 / 47, 512 rows 56 / 64, 1024 rows 84 / 73; K = 512, n =
// 2752 512 rows 48 / 57; linear, K = n = 4096 128 rows 41 / 48, 256 rows 62 / 52, 1024 rows 119 / 83;
// K = 11008, n = 4096 17 rows 35 / 53, 64 rows 62 / 55.
bool split_ok(int64_t M, int64_t K, int64_t n) {
  const int64_t groups = K / 64 * ((M + 31) / 32);
  return n * std::max<int64_t>(groups, 256) >= 6144 * 256 && qgemm_dx_slices(M, K, n) > 1;
}

// Length of the reduction that dX of the gated product walks: with two planes, both.
int64_t glu_terms(int64_t F) { return glu_two(F) ? glu_ldz(F) : 2 * F; }

// Whether a linear's G goes to dX for few rows as slices, which it adds up itself (a launch less).
// Whole backwards, us, apart / so: 4096 -> 4096 1 row 34 / 30, 96 rows (24 tiles) 42 / 39, 160 rows
// (40) 63 / 65; 1024 -> 1024 256 rows (64) 31 / 28.
bool few_dx_ok(int64_t M, int64_t K, int64_t N, int r) {
  return (M + 15) / 16 * ((r + 15) / 16) <= 64 && dx_small_ok(M, K) && !(N % 8 == 0 && split_ok(M, K, N));
}

// Backward: [dZ (gated)][G (gated: two planes of it)][its three planes][fp32 partials, of G and then of the gradients].
struct BwdWs {
  size_t dz, g, planes, part, total;
};
BwdWs bwd_ws(int64_t M, int64_t K, int64_t N, int halves, int r) {
  BwdWs w{halves == 2 ? round_up((size_t)M * glu_ldz(N) * 2) : 0, round_up((size_t)halves * halves * M * r * 2),
          round_up((size_t)3 * halves * M * g_pitch(r) * 2), 0, 0};
  size_t slices = halves == 2 ? glu_back_ws(M, N, r) : lora_skinny_ws(M, N, r);
  if (halves == 1 && few_dx_ok(M, K, N, r)) slices = std::max(slices, mx4_small_ws(M, r));
  w.part = std::max(slices, grads8_ws(M, K, N, halves, r));
  const int64_t terms = halves == 2 ? glu_terms(N) : N;
  if ((halves == 2 || N % 8 == 0) && split_ok(M, K, terms)) w.part = std::max(w.part, qgemm_dx_split_ws(M, K, terms));
  w.part = round_up(w.part);
  w.total = w.dz + w.g + w.planes + w.part;
  return w;
}

// Whether the large-tile dX product [M, K] leaves the last round of its persistent grid partly empty: the
// adapter's gradients, which need nothing of it, then take those CUs from the second stream, as in qlora_linear_bwd.
SideStream* beside_dx(int64_t M, int64_t K) {
  SideStream* sd = side_stream();
  if (!sd) return nullptr;
  const int64_t tiles = (M + 255) / 256 * ((K + 255) / 256), grid = sd->cus / 8 * 8;
  return tiles > grid && tiles % grid != 0 ? sd : nullptr;
}

// dX on `s` by `product`, then the gradients on `s` or, with sd, on the second stream beside it.
template <typename F, typename G>
int dx_and_grads(SideStream* sd, hipStream_t s, F product, G grads) {
  if (!sd) {
    QL_TRY(product());
    QL_TRY(grads(s));
    return QL_OK;
  }
  QL_TRY(hipEventRecord(sd->fork, s));
  QL_TRY(product());
  QL_TRY(hipStreamWaitEvent(sd->s, sd->fork, 0));
  QL_TRY(join_side(*sd, s, grads(sd->s)));
  return QL_OK;
}

}  // namespace

extern "C" {

size_t mx8_codes_bytes(int64_t rows, int64_t cols) {
  return matrix_ok(rows, cols, cols) ? (size_t)mx8::code_bytes(rows, cols) : 0;
}

size_t mx8_scales_bytes(int64_t rows, int64_t cols) {
  return matrix_ok(rows, cols, cols) ? (size_t)mx8::scale_bytes(rows, cols) : 0;
}

int mx8_quantize(const void* X, int x_dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales,
                 void* stream) {
  if (!X || !codes || !scales) return QL_ERR_NULL;
  if (x_dtype != QL_F32 && x_dtype != QL_BF16) return QL_ERR_DTYPE;
  if (!matrix_ok(rows, cols, ld)) return QL_ERR_SHAPE;
  if (!aligned16(X, codes, scales)) return QL_ERR_ALIGN;
  QL_TRY(launch_mx8_quant(X, x_dtype == QL_BF16, rows, cols, ld, codes, scales, (hipStream_t)stream));
  return QL_OK;
}

int mx8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint16_t* out, void* stream) {
  if (!codes || !scales || !out) return QL_ERR_NULL;
  if (!matrix_ok(rows, cols, cols)) return QL_ERR_SHAPE;
  if (!aligned16(codes, scales, out)) return QL_ERR_ALIGN;
  QL_TRY(launch_mx8_dequant(codes, scales, rows, cols, out, (hipStream_t)stream));
  return QL_OK;
}

int rms_norm_fwd(const void* X, const void* R, int x_dtype, int64_t rows, int64_t cols, const void* weight, int w_dtype,
                 float eps, void* S, uint16_t* Y, uint8_t* codes, uint8_t* scales, void* stream) {
  if (!X || !weight || (R && !S) || (!Y && !codes) || !codes != !scales) return QL_ERR_NULL;
  if ((x_dtype != QL_F32 && x_dtype != QL_BF16) || (w_dtype != QL_F32 && w_dtype != QL_BF16)) return QL_ERR_DTYPE;
  if (!matrix_ok(rows, cols, cols) || cols > kNormCols) return QL_ERR_SHAPE;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return QL_ERR_VALUE;
  if (!aligned16((const char*)X, (const char*)R, (const char*)weight, (const char*)S, Y, codes, scales)) return QL_ERR_ALIGN;
  QL_TRY(launch_norm_fwd(X, R, x_dtype == QL_BF16, rows, cols, weight, w_dtype == QL_BF16, eps, S, Y, codes, scales,
                         (hipStream_t)stream));
  return QL_OK;
}

size_t rms_norm_bwd_workspace(int64_t rows, int64_t cols) {
  return matrix_ok(rows, cols, cols) && cols <= kNormCols ? round_up(norm_bwd_ws(rows, cols)) : 0;
}

int rms_norm_bwd(const uint16_t* dY, const void* S, const void* dS, int x_dtype, int64_t rows, int64_t cols,
                 const void* weight, int w_dtype, float eps, void* dX, float* dW, void* workspace, size_t ws_bytes,
                 void* stream) {
  if (!dY || !S || !weight || (!dX && !dW)) return QL_ERR_NULL;
  if ((x_dtype != QL_F32 && x_dtype != QL_BF16) || (w_dtype != QL_F32 && w_dtype != QL_BF16)) return QL_ERR_DTYPE;
  if (!matrix_ok(rows, cols, cols) || cols > kNormCols) return QL_ERR_SHAPE;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return QL_ERR_VALUE;
  if (!aligned16(dY, (const char*)S, (const char*)dS, (const char*)weight, (const char*)dX, dW)) return QL_ERR_ALIGN;
  if (dW) {
    if (!workspace || ws_bytes < rms_norm_bwd_workspace(rows, cols)) return QL_ERR_WORKSPACE;
    if (!aligned16((const char*)workspace)) return QL_ERR_ALIGN;
  }
  QL_TRY(launch_norm_bwd(dY, S, dS, x_dtype == QL_BF16, rows, cols, weight, w_dtype == QL_BF16, eps, dX, dW,
                         (float*)workspace, (hipStream_t)stream));
  return QL_OK;
}

size_t qlora_swiglu_fwd_workspace(int64_t M, int64_t K, int64_t F, int r) {
  return glu_ok(M, K, F, r) ? fwd_ws(M, K, F, r).total : 0;
}

int qlora_swiglu_fwd(const uint16_t* X, int64_t M, int64_t K, int64_t F, const uint8_t* codes, const uint8_t* c2,
                     const float* c1, const uint16_t* L1, const uint16_t* L2, int r, float lora_scale, uint16_t* H,
                     uint16_t* T_out, uint8_t* gu_codes, uint8_t* gu_scales, void* workspace, size_t ws_bytes,
                     void* stream) {
  if (!X || !codes || !c2 || !c1 || !L1 || !L2 || !H || !gu_codes != !gu_scales) return QL_ERR_NULL;
  if (!glu_ok(M, K, F, r)) return QL_ERR_SHAPE;
  if (!aligned16(X, codes, c2, c1, L1, L2, H, T_out, gu_codes, gu_scales)) return QL_ERR_ALIGN;
  const FwdWs w = fwd_ws(M, K, F, r);
  if (!workspace || ws_bytes < w.total) return QL_ERR_WORKSPACE;
  if (!aligned16((const char*)workspace)) return QL_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  uint16_t* planes = (uint16_t*)workspace;
  float* part = (float*)((char*)workspace + w.planes);
  const int64_t pitch = w.part / sizeof(float);
  int slices = 0;
  if (few_ok(M, K, F, r)) {
    QL_TRY(launch_small_slices(X, M, K, L1, true, r, drop::Params{}, 1.0f, part, &slices, s, true));
    if (glu_decode_ok(M, K) && !gu_codes)
      QL_TRY(launch_glu_decode(X, M, K, F, codes, c2, c1, part, slices, T_out, L2, r, lora_scale, H, s));
    else
      QL_TRY(launch_glu_small(X, M, K, F, codes, c2, c1, nullptr, part, slices, T_out, L2, r, lora_scale, H, gu_codes,
                              gu_scales, s));
    return QL_OK;
  }
  for (int h = 0; h < 2; ++h)
    QL_TRY(launch_lora_slices(X, M, K, L1 + h * K * r, true, r, part + h * pitch, &slices, s));
  QL_TRY(launch_t_planes(part, pitch, slices, 2, M, r, planes, T_out, s));
  if (glu_small_ok(M, K, F))
    QL_TRY(launch_glu_small(X, M, K, F, codes, c2, c1, planes, nullptr, 0, nullptr, L2, r, lora_scale, H, gu_codes,
                            gu_scales, s));
  else
    QL_TRY(launch_glu_big(X, M, K, F, codes, c2, c1, planes, L2, r, lora_scale, H, gu_codes, gu_scales, s));
  return QL_OK;
}

size_t qlora_swiglu_bwd_workspace(int64_t M, int64_t K, int64_t F, int r) {
  return glu_ok(M, K, F, r) ? bwd_ws(M, K, F, 2, r).total : 0;
}

int qlora_swiglu_bwd(const uint8_t* x_codes, const uint8_t* x_scales, const uint16_t* dH, int64_t M, int64_t K, int64_t F,
                     const uint8_t* codes, const uint8_t* c2, const float* c1, const uint16_t* L1, const uint16_t* L2,
                     int r, float lora_scale, const uint8_t* gu_codes, const uint8_t* gu_scales, const uint16_t* T,
                     uint16_t* dX, float* dL1, float* dL2, void* workspace, size_t ws_bytes, void* stream) {
  if (!x_codes || !x_scales || !dH || !codes || !c2 || !c1 || !L1 || !L2 || !gu_codes || !gu_scales || !T || !dL1 || !dL2)
    return QL_ERR_NULL;
  if (!glu_ok(M, K, F, r)) return QL_ERR_SHAPE;
  if (!aligned16(x_codes, x_scales, dH, codes, c2, c1, L1, L2, gu_codes, gu_scales, T, dX, dL1, dL2)) return QL_ERR_ALIGN;
  const BwdWs w = bwd_ws(M, K, F, 2, r);
  if (!workspace || ws_bytes < w.total) return QL_ERR_WORKSPACE;
  if (!aligned16((const char*)workspace)) return QL_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  char* ws = (char*)workspace;
  uint16_t* dZ = (uint16_t*)ws;
  uint16_t* G = (uint16_t*)(ws + w.dz);
  uint16_t* planes = (uint16_t*)(ws + w.dz + w.g);
  float* part = (float*)(ws + w.dz + w.g + w.planes);
  int slices = 0;
  const bool two = glu_two(F);
  QL_TRY(launch_glu_back(dH, M, F, gu_codes, gu_scales, L2, r, lora_scale, dZ, part, &slices, s));
  const bool split = split_ok(M, K, glu_terms(F)), small = !split && dx_small_ok(M, K), sums = dX && small && slices <= kSmallSlices;
  if (!sums) QL_TRY(launch_low(Low{part, slices, 1.0f, G, planes, true}, 2, M, r, s));
  auto product = [&] {
    if (!dX) return hipSuccess;
    // G's planes from the product for few rows where it adds the slices up: a launch less
    if (small)
      return launch_dx_small(dZ, M, K, 2 * F, codes, c2, c1, sums ? nullptr : G, part, slices, planes, L1, r, dX, kNoDrop, s,
                             glu_ldz(F), two);
    if (split)
      return launch_qgemm_dx_split(dZ, M, K, 2 * F, codes, c2, c1, G, L1, r, dX, part, s, 2, glu_ldz(F), true, two);
    return launch_qgemm_big(true, dZ, M, K, 2 * F, codes, c2, c1, G, L1, r, 1.0f, dX, s, 2, nullptr, glu_ldz(F), true, two);
  };
  auto grads = [&](hipStream_t st) {
    return launch_grads8(Grads8{x_codes, x_scales, dH, gu_codes, gu_scales, planes, T, lora_scale, dL1, dL2}, M, K, F, 2, r,
                         part, st);
  };
  return dx_and_grads(dX && !small && !split ? beside_dx(M, K) : nullptr, s, product, grads);
}

size_t qlora_linear_bwd_mx8_workspace(int64_t M, int64_t K, int64_t N, int r) {
  return layer_ok(M, K, N, N, r) ? bwd_ws(M, K, N, 1, r).total : 0;
}

int qlora_linear_bwd_mx8(const uint8_t* x_codes, const uint8_t* x_scales, const uint16_t* dY, int64_t M, int64_t K,
                         int64_t N, const uint8_t* codes, const uint8_t* c2, const float* c1, const uint16_t* L1,
                         const uint16_t* L2, int r, float lora_scale, const uint16_t* T, uint16_t* dX, float* dL1,
                         float* dL2, void* workspace, size_t ws_bytes, void* stream) {
  if (!x_codes || !x_scales || !dY || !codes || !c2 || !c1 || !L1 || !L2 || !T || !dL1 || !dL2) return QL_ERR_NULL;
  if (!layer_ok(M, K, N, N, r)) return QL_ERR_SHAPE;
  if (!aligned16(x_codes, x_scales, dY, codes, c2, c1, L1, L2, T, dX, dL1, dL2)) return QL_ERR_ALIGN;
  const BwdWs w = bwd_ws(M, K, N, 1, r);
  if (!workspace || ws_bytes < w.total) return QL_ERR_WORKSPACE;
  if (!aligned16((const char*)workspace)) return QL_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  char* ws = (char*)workspace;
  uint16_t* G = (uint16_t*)ws;
  uint16_t* planes = (uint16_t*)(ws + w.g);
  float* part = (float*)(ws + w.g + w.planes);
  int slices = 0;
  const bool few = few_dx_ok(M, K, N, r), big = qgemm_big_ok(true, M, K, N), split = N % 8 == 0 && split_ok(M, K, N),
             small = !split && dx_small_ok(M, K);
  if (few) QL_TRY(launch_small_slices(dY, M, N, L2, false, r, kNoDrop, lora_scale, part, &slices, s));
  else QL_TRY(launch_lora_slices(dY, M, N, L2, false, r, part, &slices, s));
  if (!dX || !few) QL_TRY(launch_low(Low{part, slices, few ? 1.0f : lora_scale, G, planes, false}, 1, M, r, s));
  auto product = [&] {
    if (!dX) return hipSuccess;
    if (small)
      return launch_dx_small(dY, M, K, N, codes, c2, c1, few ? nullptr : G, part, slices, planes, L1, r, dX, kNoDrop, s);
    if (split) return launch_qgemm_dx_split(dY, M, K, N, codes, c2, c1, G, L1, r, dX, part, s);
    if (big) return launch_qgemm_big(true, dY, M, K, N, codes, c2, c1, G, L1, r, 1.0f, dX, s);
    return launch_qgemm_dx(dY, M, K, N, codes, c2, c1, G, L1, r, dX, s);
  };
  auto grads = [&](hipStream_t st) {
    return launch_grads8(Grads8{x_codes, x_scales, dY, nullptr, nullptr, planes, T, lora_scale, dL1, dL2}, M, K, N, 1, r, part,
                         st);
  };
  return dx_and_grads(dX && !small && !split && big ? beside_dx(M, K) : nullptr, s, product, grads);
}

}  // extern "C"
