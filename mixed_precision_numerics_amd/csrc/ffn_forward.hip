// Forward pass of a gated feed-forward block: both projections, the activation
// and the product in one kernel (gfx950).
//
//   [g | u] = x [Wg; Wu]^T,  y = g sigmoid(g) u
//
// Many tokens: gate_tiles.  Few tokens: gate_few, past which the weights stream
// once, which is all the time there is (ffn.hpp).
#include "ffn.hpp"

namespace amp {

hipError_t launch_gemm_swiglu(int64_t M, int64_t F, int64_t K, const void* x, int t, int64_t ldx, const void* w,
                              int64_t ldw, void* y, int64_t ldy, void* gu, int64_t ldgu, hipStream_t s) {
  ProductArgs g{};
  g.A = x; g.lda = ldx; g.B = w; g.ldb = ldw; g.M = M; g.N = F; g.K = K;
  g.C = y; g.ldc = ldy; g.gu = gu; g.ldgu = ldgu; g.splits = 1;
  return t == AMP_BF16 ? launch_gate<AMP_BF16, kOutGate>(g, s) : launch_gate<AMP_F16, kOutGate>(g, s);
}

}  // namespace amp
