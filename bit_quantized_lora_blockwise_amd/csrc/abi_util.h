// Argument checks shared by the entry points outside abi.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/qlora.h"
#include "kernels.h"

#define QL_TRY(expr)                                              \
  do {                                                            \
    const hipError_t e_ = (expr);                                 \
    if (e_ != hipSuccess) return ql_record_hip_error(e_);         \
  } while (0)

namespace qlabi {

constexpr int64_t kLim = int64_t(1) << 31;

inline size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// Every pointer given (NULL ones are skipped) on a 16-byte boundary.
template <typename... P>
inline bool aligned16(const P*... p) {
  return (((reinterpret_cast<uintptr_t>(p) & 15u) == 0) && ...);
}

// Dropout parameters from a rate, a seed and an offset; false when the rate is not in [0, 1).
inline bool drop_params(double p, uint64_t seed, uint64_t offset, drop::Params& d) {
  if (!(p >= 0.0 && p < 1.0)) return false;
  int64_t cut = (int64_t)(p * 65536.0 + 0.5);
  if (cut > 65535) cut = 65535;
  d = drop::Params{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32), (uint32_t)cut,
                   65536.0f / (float)(65536 - cut)};
  return true;
}

}  // namespace qlabi
