// Backward pass of a gated feed-forward block (gfx950).
//
//   s = sigmoid(g),  dg = dy u s (1 + g (1 - s)),  du = dy g s
//   dx = [dg | du] W,  dW = [dg | du]^T x
//
// The activation's gradient comes from the kept projections (the element-wise
// pass of amp_swiglu_backward) or out of the epilogue of the product that forms
// them again.  Both gradient products are product_tiles (ffn.hpp) on it.
#include "ffn.hpp"

namespace amp {
namespace {

// Sum of the parts of a product, in order: C[i] = sum_z part[z][i].
template <int CT>
__global__ __launch_bounds__(256) void join_parts(const float* __restrict__ part, int splits, int64_t rows, int64_t cols,
                                                  void* __restrict__ C, int64_t ldc) {
  const int64_t n = rows * cols;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    float v = part[i];
    for (int z = 1; z < splits; ++z) v += part[z * n + i];
    const int64_t at = i / cols * ldc + i % cols;
    if constexpr (CT == AMP_F32) static_cast<float*>(C)[at] = v;
    else static_cast<uint16_t*>(C)[at] = static_cast<uint16_t>(to16<CT>(v));
  }
}

// Parts of the summed dimension where the output has too few tiles for the
// machine: each at least eight steps long, their sums within the work area.
inline int parts_of(int64_t M, int64_t N, int64_t K, bool work) {
  const int64_t tiles = ceil_div(M, 128) * ceil_div(N, 128);
  if (!work || tiles >= 256) return 1;
  int64_t n = 512 / tiles;
  if (n > K / 512) n = K / 512;
  if (n > AMP_GEMM_SWIGLU_WORK / (M * N)) n = AMP_GEMM_SWIGLU_WORK / (M * N);
  return n > 1 ? static_cast<int>(n) : 1;
}

template <int ET, bool A_KC, int CT>
hipError_t gradient(ProductArgs g, float* work, hipStream_t s) {
  if (g.M == 0 || g.N == 0) return hipSuccess;
  g.splits = parts_of(g.M, g.N, g.K, work != nullptr);
  if (g.splits == 1) return launch_product<ET, A_KC, false, kOutC, CT>(g, s);
  void* const C = g.C;
  const int64_t ldc = g.ldc;
  g.C = work;
  g.ldc = g.N;
  if (hipError_t e = launch_product<ET, A_KC, false, kOutC, AMP_F32>(g, s)) return e;
  const int64_t blocks = ceil_div(g.M * g.N, 256);
  join_parts<CT><<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(work, g.splits, g.M, g.N, C, ldc);
  return hipGetLastError();
}

template <int ET>
hipError_t launch_backward(int64_t M, int64_t F, int64_t K, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                           const void* w, int64_t ldw, const void* gu, int64_t ldgu, void* dgu, int64_t lddgu, void* y,
                           int64_t ldy, void* dx, int64_t lddx, void* dw, int dwt, int64_t lddw, float* work, hipStream_t s) {
  if (M > 0 && F > 0) {
    hipError_t e;
    if (gu) {
      e = launch_swiglu_backward(dy, ET, M, F, lddy, gu, ldgu, amp_fp8_tiles{}, dgu, lddgu, amp_fp8_tiles{}, amp_fp8_tiles{},
                                 amp_fp8_tiles{}, s);
    } else {
      ProductArgs g{};
      g.A = x; g.lda = ldx; g.B = w; g.ldb = ldw; g.M = M; g.N = F; g.K = K;
      g.C = y; g.ldc = ldy; g.gu = dgu; g.ldgu = lddgu; g.dy = dy; g.lddy = lddy; g.splits = 1;
      e = launch_product<ET, true, true, kOutGrad, ET>(g, s);
    }
    if (e) return e;
  }
  if (dx) {
    ProductArgs g{};
    g.A = dgu; g.lda = lddgu; g.B = w; g.ldb = ldw; g.M = M; g.N = K; g.K = 2 * F; g.C = dx; g.ldc = lddx;
    if (hipError_t e = gradient<ET, true, ET>(g, work, s)) return e;
  }
  if (dw) {
    ProductArgs g{};
    g.A = dgu; g.lda = lddgu; g.B = x; g.ldb = ldx; g.M = 2 * F; g.N = K; g.K = M; g.C = dw; g.ldc = lddw;
    return dwt == AMP_F32 ? gradient<ET, false, AMP_F32>(g, work, s) : gradient<ET, false, ET>(g, work, s);
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_gemm_swiglu_backward(int64_t M, int64_t F, int64_t K, const void* dy, int t, int64_t lddy, const void* x,
                                       int64_t ldx, const void* w, int64_t ldw, const void* gu, int64_t ldgu, void* dgu,
                                       int64_t lddgu, void* y, int64_t ldy, void* dx, int64_t lddx, void* dw, int dwt,
                                       int64_t lddw, float* work, hipStream_t s) {
  return t == AMP_BF16 ? launch_backward<AMP_BF16>(M, F, K, dy, lddy, x, ldx, w, ldw, gu, ldgu, dgu, lddgu, y, ldy, dx, lddx,
                                                   dw, dwt, lddw, work, s)
                       : launch_backward<AMP_F16>(M, F, K, dy, lddy, x, ldx, w, ldw, gu, ldgu, dgu, lddgu, y, ldy, dx, lddx,
                                                  dw, dwt, lddw, work, s);
}

}  // namespace amp
