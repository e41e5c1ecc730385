// Transposed requantization of an FP8 checkpoint (gfx950): the wgrad operand
// of a tensor that was kept in 1x128 tiles,
//   v[r][c] = code * scale_inv * row[r] * col[c],   v^T quantized in 1x128 tiles.
// With row = rstd and col = gamma it is the normalised tensor recomputed from
// the checkpoint of the norm's input.  FP32 products, one rounding.
//
// HBM-bound: one byte in, one byte out per element (8192 x 14336 with both
// factors 46 us = 5.2 TB/s; 8192 x 4096 16 = 4.3, of which 3 are launch and tail).
// A region of odd rows reads pieces that begin at any byte, 1.9 times the bytes
// (4099 x 1111 6.9 us in a captured graph, 4096 x 1152 5.2).
#include "tiles.hpp"

namespace amp {
namespace {

struct RequantArgs {
  amp_fp8_tiles x, qt;
  int64_t rows, cols;
  const float* row; const void* col; int ct;
};

__global__ __launch_bounds__(kRegThreads) void requant_region(const RequantArgs a) {
  __shared__ RegLds<1> l;
  const Region g(a.rows, a.cols, false);
  RegRaw<1> x;
  float f[kRegRows], row[kRegRows], col[kRegCols], v[1][kRegRows][kRegCols];
#pragma unroll
  for (int i = 0; i < kRegRows; ++i) {
    const int64_t r = g.row(i);
    x.load(g, i, a.x.q + r * a.x.ldq + g.c0);
    f[i] = a.x.s[g.c0 / kTileK * a.x.lds + r];
    row[i] = a.row ? a.row[r] : 1.0f;
  }
  load_cols<kRegCols>(a.col ? elem_of(a.ct, a.col, g.c0) : nullptr, a.ct, g.c(), g.ncols, col);
  x.trim(g);
#pragma unroll
  for (int i = 0; i < kRegRows; ++i) {
    // past the end: zeros, which a scale or factor of infinity would make NaN
    const bool in = g.r() + i < g.nrows;
    decode<kRegCols>(a.x.type, x.w[i], in ? f[i] : 0.0f, v[0][i]);
    if (a.row || a.col) {
      const float r = in ? row[i] : 0.0f;
#pragma unroll
      for (int j = 0; j < kRegCols; ++j) v[0][i][j] = v[0][i][j] * r * col[j];
    }
  }
  const amp_fp8_tiles o[1] = {a.qt};
  const int64_t first[1] = {g.c0};
  reg_maxima<1>(l, g, v);
  __syncthreads();
  reg_scales<1>(l, g, o, first);
  __syncthreads();
  reg_codes<1>(l, g, o, first, v);
}

}  // namespace

hipError_t launch_requantize(const amp_fp8_tiles& x, int64_t rows, int64_t cols, const float* row, const void* col, int ct,
                             const amp_fp8_tiles& qt, hipStream_t s) {
  const int64_t most = grid_rows((cols + kTileK - 1) / kTileK) * kTileK;   // rows a launch
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    RequantArgs a{x, qt, rows - r0 < most ? rows - r0 : most, cols, row ? row + r0 : nullptr, col, ct};
    a.x.q += r0 * x.ldq;
    a.x.s += r0;
    a.qt.q += r0;
    a.qt.s += r0 / kTileK * qt.lds;
    const dim3 grid(static_cast<unsigned>((cols + kTileK - 1) / kTileK), static_cast<unsigned>((a.rows + kTileK - 1) / kTileK));
    requant_region<<<grid, kRegThreads, 0, s>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace amp
