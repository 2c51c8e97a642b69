// Internal launcher interface between the C ABI (abi.cpp) and the kernels.
// Every launcher enqueues on `s` and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"
#include "philox.h"

// Keeps a HIP error for ql_status_string and returns QL_ERR_HIP (abi.cpp).
int ql_record_hip_error(hipError_t e);

const Nf4Params& nf4_params();
const Nf4Buckets& nf4_buckets();
// Level table of a 4-bit code book: 0 NF4, 1 4-bit float (E2M1 / 6), 2 4-bit
// integer (k / 7); nullptr for any other id.
const Nf4Params* codebook_params(int codebook);

// --- encoder (encode.hip) ---------------------------------------------------
hipError_t launch_nf4_encode(const void* W, bool bf16, int64_t elems, uint8_t* codes, float* absmax,
                             hipStream_t s);
hipError_t launch_double_quant(const float* absmax, int64_t n_blocks, uint8_t* c2, float* c1, hipStream_t s);
// Both in one pass (absmax optional: may be null).
hipError_t launch_nf4_encode_dq(const void* W, bool bf16, int64_t elems, uint8_t* codes, float* absmax, uint8_t* c2,
                                float* c1, hipStream_t s);
hipError_t launch_dequant(const uint8_t* codes, const uint8_t* c2, const float* c1, int64_t elems,
                          uint16_t* out, hipStream_t s);

// --- code-book and scale-code variants (variants.hip) ------------------------
// Blockwise absmax encoder with level table p (exact division, threshold count).
hipError_t launch_q4_encode(const void* W, bool bf16, int64_t elems, const Nf4Params& p, uint8_t* codes,
                            float* absmax, hipStream_t s);
// Second-level codes over the full E4M3FN range; mean = true codes the signed
// differences from the group mean (mu[g] written), else the scales themselves.
hipError_t launch_double_quant_full(const float* absmax, int64_t n_blocks, bool mean, uint8_t* c2, float* c1,
                                    float* mu, hipStream_t s);
// Table dequantizer; mode 0: s = dec(c2) c1, 1: s = absmax, 2: s = mu + dec(c2) c1.
hipError_t launch_q4_dequant(const uint8_t* codes, int mode, const float* absmax, const uint8_t* c2,
                             const float* c1, const float* mu, int64_t elems, const Nf4Params& p, uint16_t* out,
                             hipStream_t s);

// --- skinny LoRA products (lora.hip) -----------------------------------------
// Split plan of a reduction of length R over tiles of `tiles` outputs.
struct SplitPlan {
  int splits;      // number of reduction slices
  int64_t chunk;   // reduction length per slice (multiple of 64)
};
SplitPlan plan_rowsplit(int64_t tiles, int64_t R);

// C[M, r] = A[M, R] * B, A with row stride lda, B(k, c) = L1[k][c] (b_is_kr =
// true, L1 is [R, r]) or B(k, c) = L2[c][k] (false, L2 is [r, R]).  Result
// scaled by `scale`, rounded to bf16 into out[M, r].  ws holds the fp32 partials.
size_t lora_skinny_ws(int64_t M, int64_t R, int r);
// Decode-sized T = X L1 (M <= 16, X rows 16-byte aligned, K % 64 == 0): fp32
// partial sums part[s][m][c] over S = decode_t_slices(K) <= kDecodeTSlices
// slices of the reduction.  launch_lora_skinny adds them in order s = 0..S-1 for
// such shapes, and so does the decode kernel, so T is the same on every path.
// G > 1: stacked adapters L1_g [K, r] at L1 + g K r, slices of segment g at
// part + g S M r (one launch for all).
constexpr int kDecodeTSlices = 8;
int decode_t_slices(int64_t K);
int64_t decode_t_rows(int64_t K);   // rows of K per slice (a multiple of 32)
bool decode_t_ok(int64_t M, int64_t K, const void* X, const void* L1);
hipError_t launch_lora_part(const uint16_t* X, int64_t M, int64_t K, const uint16_t* L1, int r, float* part,
                            hipStream_t s, int G = 1);
// out[i] = bf16(scale * (part[i] + part[n + i] + ...)), slices added in order.
hipError_t launch_skinny_reduce(const float* part, int slices, int64_t n, float scale, uint16_t* out, hipStream_t s);
// G = scale * (sum of the slices) [M, r] to 24 bits: three bf16 planes of pitch
// g_pitch(r) whose sum it is, and the first of them (bf16(G)) as a dense [M, r].
inline int g_pitch(int r) { return (r + 7) / 8 * 8; }
struct GPlanes {
  uint16_t* planes;     // [3][M][g_pitch(r)]
  uint16_t* dense;      // [M][r]; the first plane itself where r is its pitch
};
hipError_t launch_skinny_reduce3(const float* part, int slices, int64_t M, int r, float scale, const GPlanes& g,
                                 hipStream_t s);
hipError_t launch_lora_skinny(const uint16_t* A, int64_t M, int64_t R, int64_t lda, const uint16_t* B, bool b_is_kr,
                              int r, float scale, uint16_t* out, float* ws, hipStream_t s);

// C[p, c] = scale * sum_m A[m][p] * B[m][c] with A [M, P] (row stride lda),
// B [M, r]; stored as out[P, r] (transpose_out = false) or out[r, P] (true), fp32.
size_t lora_tn_ws(int64_t M, int64_t P, int r);
// Two such products in one launch (and their sums in one more): the first
// stored out0[P0, r], the second transposed out1_t[r, P1]; the workspace holds
// both products' partials (lora_tn_pair_ws).
size_t lora_tn_pair_ws(int64_t M, int64_t P0, int64_t P1, int r);
hipError_t launch_lora_tn_pair(const uint16_t* A0, int64_t lda0, const uint16_t* B0, int64_t P0, float scale0,
                               float* out0, const uint16_t* A1, int64_t lda1, const uint16_t* B1, int64_t P1,
                               float scale1, float* out1_t, int64_t M, int r, float* ws, hipStream_t s);
hipError_t launch_lora_tn(const uint16_t* A, int64_t lda, const uint16_t* B, int64_t M, int64_t P, int r,
                          float scale, bool transpose_out, float* out, float* ws, hipStream_t s);

// The adapter branch with dropout on its input (d.cut = 0: none) and G to 24 bits.  T and G enter
// their second products as bf16, which is what the matrix instruction takes, what the older layers
// do and, for T, what the backward is given: it costs Y 2^-9 |T| |L2| and dX 2^-9 |G| |L1|, where
// the result's own rounding costs 2^-9 of it.  dL1 is fp32 and has all of G:
//   T = bf16((D o X) L1); ws as lora_skinny_ws(M, K, r).  With `codes`, the same pass
//     also packs X (not D o X) in microscaled 4-bit; G and dY likewise
//   G = scale dY L2^T; ws as lora_skinny_ws(M, N, r)
//   dL1 [K, r] = (D o X)^T G from the planes, dL2 [r, N] = scale T^T dY, fp32; ws as
//     lora_grads3_ws(M, K, N, r).  Many rows of 16-byte pieces go to lora_grads.hip.
hipError_t launch_lora_down_drop(const uint16_t* X, int64_t M, int64_t K, const uint16_t* L1, int r,
                                 const drop::Params& d, uint16_t* T, uint8_t* codes, uint8_t* scales, float* ws,
                                 hipStream_t s);
hipError_t launch_lora_grad_in3(const uint16_t* dY, int64_t M, int64_t N, const uint16_t* L2, int r, float scale,
                                const GPlanes& G, uint8_t* codes, uint8_t* scales, float* ws, hipStream_t s);
hipError_t launch_lora_grads3(const uint16_t* X, int64_t K, const uint16_t* G, const drop::Params& d, float* dL1,
                              const uint16_t* dY, int64_t N, const uint16_t* T, float scale, float* dL2, int64_t M,
                              int r, float* ws, hipStream_t s);
size_t lora_grads3_ws(int64_t M, int64_t K, int64_t N, int r);
bool lora_grads_wide_ok(int64_t M, int64_t K, int64_t N, int r);
size_t lora_grads_wide_ws(int64_t M, int64_t K, int64_t N, int r);
hipError_t launch_lora_grads_wide(const uint16_t* X, int64_t K, const uint16_t* G, const drop::Params& d, float* dL1,
                                  const uint16_t* dY, int64_t N, const uint16_t* T, float scale, float* dL2, int64_t M,
                                  int r, float* ws, hipStream_t s);
// The sums of two such products' slices: out0 [P0, r], out1_t [r, P1] (transposed).
hipError_t launch_tn_reduce_pair(const float* part0, int splits0, int64_t P0, float scale0, float* out0,
                                 const float* part1, int splits1, int64_t P1, float scale1, float* out1_t, int r,
                                 hipStream_t s);
// Y = D o X, elementwise; X rows `ld` elements apart, Y dense (dropout.hip).
hipError_t launch_dropout(const void* X, bool bf16, int64_t rows, int64_t cols, int64_t ld, const drop::Params& d,
                          void* Y, hipStream_t s);

// --- microscaled 4-bit (mx4.hip, mx4_gemm.hip) -----------------------------------
// Quantisation along the rows of X [rows, cols] (packed rows = rows), or along its
// columns (X [len, cols], packed rows = cols); X rows `ld` elements apart.
hipError_t launch_mx4_quant(const void* X, bool bf16, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                            uint8_t* scales, hipStream_t s);
hipError_t launch_mx4_quant_t(const void* X, bool bf16, int64_t len, int64_t cols, int64_t ld, uint8_t* codes,
                              uint8_t* scales, hipStream_t s);
hipError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint16_t* out,
                              hipStream_t s);
// C[M, P] = bf16(A B^T + the adapter term), A [M, R] and B [P, R] packed.
struct Mx4Lora {
  const uint16_t* A;    // [M, r]: T (forward) or G (backward); nullptr: no adapter
  const uint16_t* B;    // forward L2 [r, P]: + scale A B; backward L1 [P, r]: + D o (A B^T)
  int r;
  bool bwd;
  float scale;          // forward only
  drop::Params d;       // backward only
};
hipError_t launch_mx4_gemm(const uint8_t* ac, const uint8_t* as, int64_t M, const uint8_t* bc, const uint8_t* bs,
                           int64_t P, int64_t R, const Mx4Lora& lora, uint16_t* C, hipStream_t s);

// The layer for few rows (mx4_small.hip): one call quantises the activations (into ac,
// as), forms T or G and multiplies.  part: mx4_small_ws bytes.  Forward: T_out may be
// nullptr.  Backward: G receives the planes alone.
bool mx4_small_ok(int64_t M, int64_t P, int64_t R, int r);   // P: columns of the result, R: of the operand
size_t mx4_small_ws(int64_t M, int r);
hipError_t launch_mx4_small_fwd(const uint16_t* X, int64_t M, int64_t K, int64_t N, const uint8_t* bc, const uint8_t* bs,
                                const uint16_t* L1, const uint16_t* L2, int r, float scale, const drop::Params& d,
                                uint16_t* Y, uint16_t* T_out, uint8_t* ac, uint8_t* as, float* part, hipStream_t s);
hipError_t launch_mx4_small_dx(const uint16_t* dY, int64_t M, int64_t K, int64_t N, const uint8_t* bc, const uint8_t* bs,
                               const uint16_t* L1, const uint16_t* L2, int r, float scale, const drop::Params& d,
                               uint16_t* dX, uint16_t* G, uint8_t* ac, uint8_t* as, float* part, hipStream_t s);
// The forward's T and the backward's G alone (same bits).
hipError_t launch_mx4_small_t(const uint16_t* X, int64_t M, int64_t K, const uint16_t* L1, int r, const drop::Params& d,
                              uint16_t* T, float* part, hipStream_t s);
hipError_t launch_mx4_small_g(const uint16_t* dY, int64_t M, int64_t N, const uint16_t* L2, int r, float scale,
                              uint16_t* G, float* part, hipStream_t s);
// fp32 slices (part: mx4_small_ws bytes) of scale (D o A) B (L1, b_is_kr) or scale A B^T (L2), to be
// added in order.
hipError_t launch_small_slices(const uint16_t* A, int64_t M, int64_t R, const uint16_t* B, bool b_is_kr, int r,
                               const drop::Params& d, float scale, float* part, int* slices, hipStream_t s);

// --- adapter merge (merge.hip) ---------------------------------------------
// W[n][k] = bf16(W'[n][k] + scale * sum_c L1[k][c] L2[c][n]), W' the bf16
// dequantised base; W [N, K], K a multiple of 64.
hipError_t launch_merge(const uint8_t* codes, const uint8_t* c2, const float* c1, int64_t N, int64_t K,
                        const uint16_t* L1, const uint16_t* L2, int r, float scale, uint16_t* W, hipStream_t s);

// --- adapter optimizer (adamw.hip) -------------------------------------------
// One AdamW step over n fp32 weights (decoupled decay), optional bf16 copy.
hipError_t launch_adamw(float* param, float* exp_avg, float* exp_avg_sq, const float* grad, uint16_t* param_bf16,
                        int64_t n, float lr, float beta1, float beta2, float eps, float weight_decay, int64_t step,
                        hipStream_t s);

// --- quantised GEMMs (gemm_big.hip, gemm.hip, decode.hip) ----------------------
// Y[M, N] = bf16(X W'^T + scale * T L2) for small M (M <= 16), streaming the
// packed weight once (training-sized M: launch_qgemm_big below).
hipError_t launch_qgemv_fwd(const uint16_t* X, int64_t M, int64_t K, int64_t N, const uint8_t* codes,
                            const uint8_t* c2, const float* c1, const uint16_t* T, const uint16_t* L2, int r,
                            float scale, uint16_t* Y, hipStream_t s);
// Same, with T = bf16(sum over s of Tpart[s]) formed by the kernel from the S
// fp32 slices of launch_lora_part (r % 4 == 0, Tpart 16-byte aligned); T_out
// (optional) receives that T.
// Stacked linears at decode size: G segments of N rows of one packed matrix
// [G N, K] sharing X, each with its own T (formed from the slices of
// launch_lora_part(..., G)) and L2_g [r, N] (at L2 + g r N); Y [M, G N].  Only
// for X that fits the kernel's LDS (M K <= 16384) and N % 16 == 0.
bool qgemv_group_ok(int64_t M, int64_t K, int64_t N, int G);
hipError_t launch_qgemv_group_tpart(const uint16_t* X, int64_t M, int64_t K, int64_t N, int G, const uint8_t* codes,
                                    const uint8_t* c2, const float* c1, const float* Tpart, int S, uint16_t* T_out,
                                    const uint16_t* L2, int r, float scale, uint16_t* Y, hipStream_t s);
hipError_t launch_qgemv_fwd_tpart(const uint16_t* X, int64_t M, int64_t K, int64_t N, const uint8_t* codes,
                                  const uint8_t* c2, const float* c1, const float* Tpart, int S, uint16_t* T_out,
                                  const uint16_t* L2, int r, float scale, uint16_t* Y, hipStream_t s);
// The same decode forward with T formed inside the one launch (no separate
// partial-sum launch): M * K * 2 <= 32 KB, r % 4 == 0, r <= 64.  part: S M r
// fp32 (16-byte aligned); sync: qgemv_fused_sync_bytes(M, r) bytes (16-byte
// aligned) of flags and T records, holding anything but data tagged with
// `epoch`, which must differ from every earlier call's epoch on the same memory
// (in its low 32 bits too, which must not be 0); spins bounds each wave's wait
// (past it the wave forms T's slices itself, same bits).
bool qgemv_fused_ok(int64_t M, int64_t K, int r);
size_t qgemv_fused_sync_bytes(int64_t M, int r);
hipError_t launch_qgemv_fwd_fused(const uint16_t* X, int64_t M, int64_t K, int64_t N, const uint8_t* codes,
                                  const uint8_t* c2, const float* c1, const uint16_t* L1, int r, float* part,
                                  void* sync, uint64_t epoch, uint32_t spins, uint16_t* T_out,
                                  const uint16_t* L2, float scale, uint16_t* Y, hipStream_t s);
// Large-tile (256 x 256) versions of both GEMMs: dx = false computes the forward
// (A = X, LA = T, LB = L2, C = Y), dx = true the dX product (A = dY, LA = G,
// LB = L1, C = dX).  qgemm_big_ok says whether the shapes qualify.  nseg > 1:
// W [N, K] is nseg matrices of N / nseg rows stacked (N / nseg a multiple of
// 256), each with its own adapter: LA holds nseg [M, r] blocks, LB nseg L2
// [r, N / nseg] (fwd) or L1 [K, r] (dX) blocks.  d (dX, nseg = 1): dropout of the
// adapter term, dX = bf16(dY W' + D o (G L1^T)).
bool qgemm_big_ok(bool dx, int64_t M, int64_t K, int64_t N);
hipError_t launch_qgemm_big(bool dx, const uint16_t* A, int64_t M, int64_t K, int64_t N, const uint8_t* codes,
                            const uint8_t* c2, const float* c1, const uint16_t* LA, const uint16_t* LB, int r,
                            float scale, uint16_t* C, hipStream_t s, int nseg = 1,
                            const drop::Params* d = nullptr);
// The same two GEMMs with a bf16 weight W [N, K] in place of the packed one
// (LoRA over a bf16 base): dx = false Y = bf16(X W^T + scale T L2), dx = true
// dX = bf16(dY W + G L1^T).  bgemm_ok says whether the shapes qualify.
bool bgemm_ok(bool dx, int64_t M, int64_t K, int64_t N);
hipError_t launch_bgemm_big(bool dx, const uint16_t* A, int64_t M, int64_t K, int64_t N, const uint16_t* W,
                            const uint16_t* LA, const uint16_t* LB, int r, float scale, uint16_t* C, hipStream_t s);
// dX[M, K] = bf16(dY W' + G L1^T), d as above
hipError_t launch_qgemm_dx(const uint16_t* dY, int64_t M, int64_t K, int64_t N, const uint8_t* codes,
                           const uint8_t* c2, const float* c1, const uint16_t* G, const uint16_t* L1, int r,
                           uint16_t* dX, hipStream_t s, const drop::Params* d = nullptr);
// The NF4 layer with dropout for few rows (gemm_small.hip).  Forward: Y = bf16(X W'^T + scale (T L2))
// from T, or with T = nullptr from its slices Tp (S of them), added here; T_out then receives it.
bool fwd_small_ok(int64_t M, int64_t N);
hipError_t launch_fwd_small(const uint16_t* X, int64_t M, int64_t K, int64_t N, const uint8_t* codes, const uint8_t* c2,
                            const float* c1, const uint16_t* T, const float* Tp, int S, uint16_t* T_out,
                            const uint16_t* L2, int r, float scale, uint16_t* Y, hipStream_t s);
// dX = bf16(dY W' + D o (G L1^T)) from G, or with G = nullptr from its slices Gp (S of them), added
// here; `planes` then receives it to 24 bits.
bool dx_small_ok(int64_t M, int64_t K);
hipError_t launch_dx_small(const uint16_t* dY, int64_t M, int64_t K, int64_t N, const uint8_t* codes, const uint8_t* c2,
                           const float* c1, const uint16_t* G, const float* Gp, int S, uint16_t* planes,
                           const uint16_t* L1, int r, uint16_t* dX, const drop::Params& d, hipStream_t s);
