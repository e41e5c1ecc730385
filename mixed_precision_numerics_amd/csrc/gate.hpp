// The gate of a gated activation, shared by the element-wise passes and the
// GEMM epilogues.
#pragma once
#include "common.hpp"

namespace amp {
namespace {

// s = 1 / (1 + e), e = exp(-g), from the hardware's exponential and
// reciprocal (each within an ulp; the scaled argument's roundings grow with
// |g|, so that e is off by up to |g| 2^-22 and s by that times 1 - s).  Below g
// = -87 s leaves the normal range and may be 0, as e overflows at -89.  g = -inf
// gives s = 0 and, as in the formula, 0 * inf = NaN for g s.  Where e overflows
// s is 0 and e s a NaN, of which the minimum makes 1 (a NaN g leaves one in s).
struct Gate { float s, om; };   // s and 1 - s
__device__ __forceinline__ Gate gate(float g) {
  const float e = __builtin_amdgcn_exp2f(g * -1.4426950408889634f);
  const float s = __builtin_amdgcn_rcpf(1.0f + e);
  return {s, __builtin_fminf(e * s, 1.0f)};
}

}  // namespace
}  // namespace amp
