// Backward pass of a gated feed-forward block (gfx950).
//
//   s = sigmoid(g),  dg = dy u s (1 + g (1 - s)),  du = dy g s
//   dx = [dg | du] W,  dW = [dg | du]^T x
//
// The activation's gradient comes from the kept projections (the element-wise
// pass of amp_swiglu_backward) or out of the epilogue of the product that forms
// them again.  The two gradient products on it are one launch.
//
// dg and du are rounded to the operands' 16 bits before the two products: they
// are what the matrix cores multiply, and a second part for what the rounding
// leaves would double the products.  That rounding is all that sets dx and dw apart
// from products of FP32 gradients: relative to those 2.6e-3 in BF16 and 3.2e-4 in
// F16 over whole outputs, and 1e-4 and 2e-5 relative to products of the rounded ones.
//
// Bound by the matrix cores: 8192 x 4096 x 14336 BF16 from kept projections 3.05 ms,
// of which the element-wise pass is 0.18 and the products run at 1.35 PFLOP/s;
// 4000 x 5120 x 10240 with them formed again 2.0 ms, 0.68 of it for forming them.
// Small ones are bound by the ends of three short launches: 777 x 512 x 2048 F16 25 us
// (5.3 + 16.6 + 4.8 one by one).
#include "ffn.hpp"

namespace amp {
namespace {

// Sum of the parts of a product, in order: C[i] = sum_z part[z][i].  Eight loads are
// under way at a time (79 parts of 45 x 64: 18.6 -> 6.5 us).
template <int CT>
__global__ __launch_bounds__(256) void join_parts(const float* __restrict__ part, int splits, int64_t rows, int64_t cols,
                                                  void* __restrict__ C, int64_t ldc) {
  const int64_t n = rows * cols;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    float v = part[i];
    int z = 1;
    for (; z + 8 <= splits; z += 8) {
      float p[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) p[k] = part[(z + k) * n + i];
#pragma unroll
      for (int k = 0; k < 8; ++k) v += p[k];
    }
    for (; z < splits; ++z) v += part[z * n + i];
    const int64_t at = i / cols * ldc + i % cols;
    if constexpr (CT == AMP_F32) static_cast<float*>(C)[at] = v;
    else static_cast<uint16_t*>(C)[at] = static_cast<uint16_t>(to16<CT>(v));
  }
}

template <int ET>
hipError_t join(const ProductArgs& g, const float* part, void* C, int64_t ldc, int ct, hipStream_t s) {
  const int64_t blocks = ceil_div(g.M * g.N, 256);
  const unsigned grid = static_cast<unsigned>(blocks < 4096 ? blocks : 4096);
  if (ct == AMP_F32) join_parts<AMP_F32><<<grid, 256, 0, s>>>(part, g.splits, g.M, g.N, C, ldc);
  else join_parts<ET><<<grid, 256, 0, s>>>(part, g.splits, g.M, g.N, C, ldc);
  return hipGetLastError();
}

// dx = dgu w and dw = dgu^T x (either may be absent, M * N == 0).
template <int ET>
hipError_t gradients(ProductArgs gx, ProductArgs gw, int ct, float* work, hipStream_t s) {
  const bool dx = gx.C && gx.M > 0 && gx.N > 0, dw = gw.C && gw.M > 0 && gw.N > 0;
  if (!dx && !dw) return hipSuccess;
  if (!dx) gx.M = gx.N = 0;
  if (!dw) gw.M = gw.N = 0;
  const bool fast = (!dx || (direct_operand(gx.A, gx.lda, true, gx.M) && direct_operand(gx.B, gx.ldb, false, gx.N))) &&
                    (!dw || (direct_operand(gw.A, gw.lda, false, gw.M) && direct_operand(gw.B, gw.ldb, false, gw.N)));
  const GradientForm f = gradient_form(gx.M, gx.N, gx.K, gw.M, gw.N, gw.K, fast, work ? AMP_GEMM_SWIGLU_WORK : 0);
  gx.splits = f.split_x;
  gw.splits = f.split_w;
  const ProductArgs x0 = gx, w0 = gw;      // where the results go
  gx.out32 = gx.splits > 1;
  if (gx.splits > 1) { gx.C = work; gx.ldc = gx.N; }
  gw.out32 = gw.splits > 1 || ct == AMP_F32;
  if (gw.splits > 1) { gw.C = work + (gx.splits > 1 ? gx.splits * gx.M * gx.N : 0); gw.ldc = gw.N; }
  const int64_t edge = f.wide ? 256 : 128;
  const uint32_t nx = static_cast<uint32_t>(tiles_of(gx.M, gx.N, edge) * gx.splits), nw = static_cast<uint32_t>(tiles_of(gw.M, gw.N, edge) * gw.splits);
  if (f.wide) gradient_tiles<ET, 4, 4, true><<<nx + nw, 256, 0, s>>>(gx, gw, nx, nw, f.dx_first);
  else if (fast) gradient_tiles<ET, 2, 2, true><<<nx + nw, 256, 0, s>>>(gx, gw, nx, nw, f.dx_first);
  else gradient_tiles<ET, 2, 2, false><<<nx + nw, 256, 0, s>>>(gx, gw, nx, nw, f.dx_first);
  if (hipError_t e = hipGetLastError()) return e;
  if (gx.splits > 1)
    if (hipError_t e = join<ET>(gx, static_cast<const float*>(gx.C), x0.C, x0.ldc, ET, s)) return e;
  return gw.splits > 1 ? join<ET>(gw, static_cast<const float*>(gw.C), w0.C, w0.ldc, ct, s) : hipSuccess;
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
      e = launch_gate<ET, kOutGrad>(g, s);
    }
    if (e) return e;
  }
  ProductArgs gx{}, gw{};
  gx.A = dgu; gx.lda = lddgu; gx.B = w; gx.ldb = ldw; gx.M = M; gx.N = K; gx.K = 2 * F; gx.C = dx; gx.ldc = lddx;
  gw.A = dgu; gw.lda = lddgu; gw.B = x; gw.ldb = ldx; gw.M = 2 * F; gw.N = K; gw.K = M; gw.C = dw; gw.ldc = lddw;
  return gradients<ET>(gx, gw, dwt, work, s);
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
