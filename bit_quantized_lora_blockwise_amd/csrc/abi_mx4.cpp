// Entry points of the microscaled 4-bit layer and of the adapter dropout: argument
// checks, workspace layout and dispatch.  Contracts: include/qlora.h.
#include <algorithm>

#include "abi_util.h"
#include "mx4.h"
#include "side_stream.h"

namespace {

using namespace qlabi;

constexpr int64_t kMaxElems = int64_t(1) << 40;

bool matrix_ok(int64_t rows, int64_t cols, int64_t ld) {
  return rows > 0 && cols > 0 && rows < kLim && cols < kLim && ld >= cols && ld <= kMaxElems / rows;
}

// Layer sizes: X, Y and their gradients, the packed activations and the packed
// weight, the adapters, T and each plane of G below 2^31 bytes (the kernels' offsets are
// 32-bit; G's three planes together may pass it).
bool layer_ok(int64_t M, int64_t K, int64_t N, int r) {
  return M > 0 && K > 0 && N > 0 && M < kLim && K < kLim && N < kLim && r >= 1 && r <= 64 && M <= kLim / 2 / K &&
         M <= kLim / 2 / N && M < kLim / 2 / r && K < kLim / 2 / r && N < kLim / 2 / r && M * K * 2 < kLim &&
         M * N * 2 < kLim && mx4::padded(K) <= kLim / N && mx4::padded(N) <= kLim / K &&
         mx4::code_bytes(N, K) < kLim && mx4::code_bytes(K, N) < kLim && mx4::code_bytes(M, K) < kLim &&
         mx4::code_bytes(M, N) < kLim;
}

// [packed activations: codes, scales][T or the three planes of G][dense G][T of a backward without one][fp32 partials]
struct Ws {
  size_t codes, scales, low, dense, t, part, total;
};
// The slices of T = (D o X) L1 of the microscaled layer; of G with K and N exchanged.
size_t slices_ws(int64_t M, int64_t K, int64_t N, int r) {
  return mx4_small_ok(M, N, K, r) ? mx4_small_ws(M, r) : lora_skinny_ws(M, K, r);
}
Ws fwd_ws(int64_t M, int64_t K, int64_t N, int r) {
  Ws w{round_up(mx4::code_bytes(M, K)), round_up(mx4::scale_bytes(M, K)), round_up((size_t)M * r * 2), 0, 0,
       round_up(slices_ws(M, K, N, r)), 0};
  w.total = w.codes + w.scales + w.low + w.part;
  return w;
}
// Whether the NF4 layer with dropout forms T and G as slices that its products add up (a launch
// less each): while the rank-r product has few 16 x 16 tiles.  Whole forwards, us, slices / sums of
// their own: 64 rows of rank 64 (16 tiles) 11008 -> 4096 42 / 46, 128 rows of rank 36 (24) 8576 -> 631
// 32 / 36, 192 rows (36) 38 / 37, 128 rows of rank 64 (32) 11008 -> 4096 58 / 57, 256 rows (64) 91 / 80.
bool few_ok(int64_t M, int64_t K, int64_t N, int r) {
  return (M + 15) / 16 * ((r + 15) / 16) <= 24 && layer_ok(M, K, N, r);
}

// packed = false: the backward over another base, which multiplies the bf16 gradient; its
// slices are counted for every p
Ws bwd_ws(int64_t M, int64_t K, int64_t N, int r, bool packed) {
  Ws w{packed ? round_up(mx4::code_bytes(M, N)) : 0, packed ? round_up(mx4::scale_bytes(M, N)) : 0,
       round_up((size_t)3 * M * g_pitch(r) * 2), r == g_pitch(r) ? 0 : round_up((size_t)M * r * 2),
       round_up((size_t)M * r * 2), 0, 0};
  const size_t slices = packed ? std::max(slices_ws(M, K, N, r), slices_ws(M, N, K, r))
                               : std::max({lora_skinny_ws(M, N, r), lora_skinny_ws(M, K, r),
                                           few_ok(M, K, N, r) ? mx4_small_ws(M, r) : 0});
  w.part = round_up(std::max(slices, lora_grads3_ws(M, K, N, r)));
  w.total = w.codes + w.scales + w.low + w.dense + w.t + w.part;
  return w;
}

}  // namespace

extern "C" {

size_t mx4_codes_bytes(int64_t rows, int64_t cols) {
  return matrix_ok(rows, cols, cols) ? (size_t)mx4::code_bytes(rows, cols) : 0;
}

size_t mx4_scales_bytes(int64_t rows, int64_t cols) {
  return matrix_ok(rows, cols, cols) ? (size_t)mx4::scale_bytes(rows, cols) : 0;
}

int mx4_quantize(const void* X, int x_dtype, int64_t rows, int64_t cols, int64_t ld, int transpose, uint8_t* codes,
                 uint8_t* scales, void* stream) {
  if (!X || !codes || !scales) return QL_ERR_NULL;
  if (x_dtype != QL_F32 && x_dtype != QL_BF16) return QL_ERR_DTYPE;
  if (!matrix_ok(rows, cols, ld)) return QL_ERR_SHAPE;
  if (!aligned16(X, codes, scales)) return QL_ERR_ALIGN;
  if (transpose)
    QL_TRY(launch_mx4_quant_t(X, x_dtype == QL_BF16, rows, cols, ld, codes, scales, (hipStream_t)stream));
  else
    QL_TRY(launch_mx4_quant(X, x_dtype == QL_BF16, rows, cols, ld, codes, scales, (hipStream_t)stream));
  return QL_OK;
}

int mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint16_t* out,
                   void* stream) {
  if (!codes || !scales || !out) return QL_ERR_NULL;
  if (!matrix_ok(rows, cols, cols)) return QL_ERR_SHAPE;
  if (!aligned16(codes, scales, out)) return QL_ERR_ALIGN;
  QL_TRY(launch_mx4_dequant(codes, scales, rows, cols, out, (hipStream_t)stream));
  return QL_OK;
}

int mx4_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M, const uint8_t* b_codes,
               const uint8_t* b_scales, int64_t N, int64_t K, uint16_t* C, void* stream) {
  if (!a_codes || !a_scales || !b_codes || !b_scales || !C) return QL_ERR_NULL;
  if (!layer_ok(M, K, N, 1)) return QL_ERR_SHAPE;
  if (!aligned16(a_codes, a_scales, b_codes, b_scales, C)) return QL_ERR_ALIGN;
  QL_TRY(launch_mx4_gemm(a_codes, a_scales, M, b_codes, b_scales, N, K, Mx4Lora{}, C, (hipStream_t)stream));
  return QL_OK;
}

int lora_dropout(const void* X, int x_dtype, int64_t rows, int64_t cols, int64_t ld, double p, uint64_t seed,
                 uint64_t offset, void* Y, void* stream) {
  if (!X || !Y) return QL_ERR_NULL;
  if (x_dtype != QL_F32 && x_dtype != QL_BF16) return QL_ERR_DTYPE;
  if (!matrix_ok(rows, cols, ld)) return QL_ERR_SHAPE;
  drop::Params d;
  if (!drop_params(p, seed, offset, d)) return QL_ERR_VALUE;
  if (!aligned16(X, Y)) return QL_ERR_ALIGN;
  QL_TRY(launch_dropout(X, x_dtype == QL_BF16, rows, cols, ld, d, Y, (hipStream_t)stream));
  return QL_OK;
}

size_t mx4_linear_fwd_workspace(int64_t M, int64_t K, int64_t N, int r) {
  return layer_ok(M, K, N, r) ? fwd_ws(M, K, N, r).total : 0;
}

int mx4_linear_fwd(const uint16_t* X, int64_t M, int64_t K, int64_t N, const uint8_t* codes, const uint8_t* scales,
                   const uint16_t* L1, const uint16_t* L2, int r, float lora_scale, double p, uint64_t seed,
                   uint64_t offset, uint16_t* Y, uint16_t* T_out, void* workspace, size_t ws_bytes, void* stream) {
  if (!X || !codes || !scales || !L1 || !L2 || !Y) return QL_ERR_NULL;
  if (!layer_ok(M, K, N, r)) return QL_ERR_SHAPE;
  drop::Params d;
  if (!drop_params(p, seed, offset, d)) return QL_ERR_VALUE;
  if (!aligned16(X, codes, scales, L1, L2, Y, T_out)) return QL_ERR_ALIGN;
  const Ws w = fwd_ws(M, K, N, r);
  if (!workspace || ws_bytes < w.total) return QL_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QL_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* ac = (uint8_t*)workspace;
  uint8_t* as = ac + w.codes;
  uint16_t* T = T_out ? T_out : (uint16_t*)(as + w.scales);
  float* part = (float*)(as + w.scales + w.low);
  if (mx4_small_ok(M, N, K, r)) {
    QL_TRY(launch_mx4_small_fwd(X, M, K, N, codes, scales, L1, L2, r, lora_scale, d, Y, T_out, ac, as, part, s));
    return QL_OK;
  }
  QL_TRY(launch_lora_down_drop(X, M, K, L1, r, d, T, ac, as, part, s));
  QL_TRY(launch_mx4_gemm(ac, as, M, codes, scales, N, K, Mx4Lora{T, L2, r, false, lora_scale, drop::Params{}}, Y, s));
  return QL_OK;
}

size_t mx4_linear_bwd_workspace(int64_t M, int64_t K, int64_t N, int r) {
  return layer_ok(M, K, N, r) ? bwd_ws(M, K, N, r, true).total : 0;
}

int mx4_linear_bwd(const uint16_t* X, const uint16_t* dY, int64_t M, int64_t K, int64_t N, const uint8_t* codes_t,
                   const uint8_t* scales_t, const uint16_t* L1, const uint16_t* L2, int r, float lora_scale, double p,
                   uint64_t seed, uint64_t offset, const uint16_t* T, uint16_t* dX, float* dL1, float* dL2,
                   void* workspace, size_t ws_bytes, void* stream) {
  if (!X || !dY || !codes_t || !scales_t || !L1 || !L2 || !dL1 || !dL2) return QL_ERR_NULL;
  if (!layer_ok(M, K, N, r)) return QL_ERR_SHAPE;
  drop::Params d;
  if (!drop_params(p, seed, offset, d)) return QL_ERR_VALUE;
  if (!aligned16(X, dY, codes_t, scales_t, L1, L2, T, dX, dL1, dL2)) return QL_ERR_ALIGN;
  const Ws w = bwd_ws(M, K, N, r, true);
  if (!workspace || ws_bytes < w.total) return QL_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QL_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* ac = (uint8_t*)workspace;
  uint8_t* as = ac + w.codes;
  uint8_t* low = as + w.scales;
  const GPlanes G{(uint16_t*)low, (uint16_t*)(w.dense ? low + w.low : low)};
  uint16_t* Tw = (uint16_t*)(low + w.low + w.dense);
  float* part = (float*)((uint8_t*)Tw + w.t);
  const bool small = mx4_small_ok(M, K, N, r);
  if (!T) {
    if (mx4_small_ok(M, N, K, r)) QL_TRY(launch_mx4_small_t(X, M, K, L1, r, d, Tw, part, s));
    else QL_TRY(launch_lora_down_drop(X, M, K, L1, r, d, Tw, nullptr, nullptr, part, s));
    T = Tw;
  }
  if (dX && small) {
    QL_TRY(launch_mx4_small_dx(dY, M, K, N, codes_t, scales_t, L1, L2, r, lora_scale, d, dX, G.planes, ac, as, part, s));
  } else if (small) {
    QL_TRY(launch_mx4_small_g(dY, M, N, L2, r, lora_scale, G.planes, part, s));
  } else {
    QL_TRY(launch_lora_grad_in3(dY, M, N, L2, r, lora_scale, G, dX ? ac : nullptr, as, part, s));
    if (dX) QL_TRY(launch_mx4_gemm(ac, as, M, codes_t, scales_t, K, N, Mx4Lora{G.dense, L1, r, true, 1.0f, d}, dX, s));
  }
  QL_TRY(launch_lora_grads3(X, K, G.planes, d, dL1, dY, N, T, lora_scale, dL2, M, r, part, s));
  return QL_OK;
}

// ---- dropout on the adapter of the NF4 layer ------------------------------------
size_t qlora_linear_fwd_dropout_workspace(int64_t M, int64_t K, int64_t N, int r) {
  const size_t plain = qlora_linear_fwd_workspace(M, K, N, r);
  return plain == 0 ? 0 : std::max(plain, round_up((size_t)M * r * 2) + (few_ok(M, K, N, r) ? mx4_small_ws(M, r) : 0));
}

int qlora_linear_fwd_dropout(const uint16_t* X, int64_t M, int64_t K, int64_t N, const uint8_t* codes,
                             const uint8_t* c2, const float* c1, const uint16_t* L1, const uint16_t* L2, int r,
                             float lora_scale, double p, uint64_t seed, uint64_t offset, uint16_t* Y, uint16_t* T_out,
                             void* workspace, size_t ws_bytes, void* stream) {
  if (!X || !codes || !c2 || !c1 || !L1 || !L2 || !Y) return QL_ERR_NULL;
  const size_t need = qlora_linear_fwd_dropout_workspace(M, K, N, r);
  if (need == 0) return QL_ERR_SHAPE;
  drop::Params d;
  if (!drop_params(p, seed, offset, d)) return QL_ERR_VALUE;
  if (d.cut == 0)
    return qlora_linear_fwd(X, M, K, N, codes, c2, c1, L1, L2, r, lora_scale, Y, T_out, workspace, ws_bytes, stream);
  if (!aligned16(X, codes, c2, c1, L1, L2, Y, T_out)) return QL_ERR_ALIGN;
  if (!workspace || ws_bytes < need) return QL_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QL_ERR_ALIGN;
  uint16_t* T = T_out ? T_out : (uint16_t*)workspace;
  float* part = (float*)((char*)workspace + round_up((size_t)M * r * 2));
  hipStream_t s = (hipStream_t)stream;
  if (few_ok(M, K, N, r)) {
    int S = 0;
    QL_TRY(launch_small_slices(X, M, K, L1, true, r, d, d.scale, part, &S, s));
    if (fwd_small_ok(M, N)) {
      QL_TRY(launch_fwd_small(X, M, K, N, codes, c2, c1, nullptr, part, S, T_out, L2, r, lora_scale, Y, s));
      return QL_OK;
    }
    if (M <= 16 && r % 4 == 0) {
      QL_TRY(launch_qgemv_fwd_tpart(X, M, K, N, codes, c2, c1, part, S, T_out, L2, r, lora_scale, Y, s));
      return QL_OK;
    }
    QL_TRY(launch_skinny_reduce(part, S, M * r, 1.0f, T, s));
  } else {
    QL_TRY(launch_lora_down_drop(X, M, K, L1, r, d, T, nullptr, nullptr, part, s));
    if (fwd_small_ok(M, N)) {
      QL_TRY(launch_fwd_small(X, M, K, N, codes, c2, c1, T, nullptr, 0, nullptr, L2, r, lora_scale, Y, s));
      return QL_OK;
    }
  }
  return qlora_linear_fwd_t(X, M, K, N, codes, c2, c1, T, L2, r, lora_scale, Y, stream);
}

size_t qlora_linear_bwd_dropout_workspace(int64_t M, int64_t K, int64_t N, int r) {
  return qlora_linear_bwd_workspace(M, K, N, r) == 0 ? 0 : bwd_ws(M, K, N, r, false).total;
}

int qlora_linear_bwd_dropout(const uint16_t* X, const uint16_t* dY, int64_t M, int64_t K, int64_t N,
                             const uint8_t* codes, const uint8_t* c2, const float* c1, const uint16_t* L1,
                             const uint16_t* L2, int r, float lora_scale, double p, uint64_t seed, uint64_t offset,
                             const uint16_t* T, uint16_t* dX, float* dL1, float* dL2, void* workspace,
                             size_t ws_bytes, void* stream) {
  if (!X || !dY || !codes || !c2 || !c1 || !L1 || !L2 || !dL1 || !dL2) return QL_ERR_NULL;
  if (qlora_linear_bwd_workspace(M, K, N, r) == 0) return QL_ERR_SHAPE;
  drop::Params d;
  if (!drop_params(p, seed, offset, d)) return QL_ERR_VALUE;
  if (!aligned16(X, dY, codes, c2, c1, L1, L2, T, dX, dL1, dL2)) return QL_ERR_ALIGN;
  const Ws w = bwd_ws(M, K, N, r, false);
  if (!workspace || ws_bytes < w.total) return QL_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QL_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* low = (uint8_t*)workspace;
  const GPlanes G{(uint16_t*)low, (uint16_t*)(w.dense ? low + w.low : low)};
  uint16_t* Tw = (uint16_t*)(low + w.low + w.dense);
  float* part = (float*)((uint8_t*)Tw + w.t);
  const bool few = d.cut != 0 && few_ok(M, K, N, r), small = dx_small_ok(M, K);
  int S = 0;
  if (!T) {
    if (few) {
      QL_TRY(launch_small_slices(X, M, K, L1, true, r, d, d.scale, part, &S, s));
      QL_TRY(launch_skinny_reduce(part, S, M * r, 1.0f, Tw, s));
    } else {
      QL_TRY(launch_lora_down_drop(X, M, K, L1, r, d, Tw, nullptr, nullptr, part, s));
    }
    T = Tw;
  }
  if (few && small) {
    QL_TRY(launch_small_slices(dY, M, N, L2, false, r, d, lora_scale, part, &S, s));
    if (dX)
      QL_TRY(launch_dx_small(dY, M, K, N, codes, c2, c1, nullptr, part, S, G.planes, L1, r, dX, d, s));
    else
      QL_TRY(launch_skinny_reduce3(part, S, M, r, 1.0f, G, s));
  } else {
    QL_TRY(launch_lora_grad_in3(dY, M, N, L2, r, lora_scale, G, nullptr, nullptr, part, s));
    SideStream* sd = dX && !(d.cut && small) && qgemm_big_ok(true, M, K, N) ? side_stream() : nullptr;
    const int64_t tiles = (M + 255) / 256 * ((K + 255) / 256), grid = sd ? sd->cus / 8 * 8 : 1;
    if (sd && tiles > grid && tiles % grid != 0) {
      // As in qlora_linear_bwd: the gradients take the CUs that dX's last round leaves idle.  2048 rows
      // 22016 -> 8192 698 us, 717 one after the other, 11008 -> 4096 253 and 267; 4096 rows of it 428 and 425.
      // (The microscaled backward stays in order: 196 us against 189 at 4096 rows 11008 -> 4096.)
      QL_TRY(hipEventRecord(sd->fork, s));
      QL_TRY(launch_qgemm_big(true, dY, M, K, N, codes, c2, c1, G.dense, L1, r, 1.0f, dX, s, 1, &d));
      QL_TRY(hipStreamWaitEvent(sd->s, sd->fork, 0));
      const hipError_t e = launch_lora_grads3(X, K, G.planes, d, dL1, dY, N, T, lora_scale, dL2, M, r, part, sd->s);
      QL_TRY(join_side(*sd, s, e));
      return QL_OK;
    }
    if (dX) {
      if (d.cut && small)
        QL_TRY(launch_dx_small(dY, M, K, N, codes, c2, c1, G.dense, nullptr, 0, nullptr, L1, r, dX, d, s));
      else if (qgemm_big_ok(true, M, K, N))
        QL_TRY(launch_qgemm_big(true, dY, M, K, N, codes, c2, c1, G.dense, L1, r, 1.0f, dX, s, 1, &d));
      else
        QL_TRY(launch_qgemm_dx(dY, M, K, N, codes, c2, c1, G.dense, L1, r, dX, s, &d));
    }
  }
  QL_TRY(launch_lora_grads3(X, K, G.planes, d, dL1, dY, N, T, lora_scale, dL2, M, r, part, s));
  return QL_OK;
}

}  // extern "C"
