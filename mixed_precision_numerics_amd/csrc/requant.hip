// Transposed requantization of an FP8 checkpoint (gfx950): the wgrad operand
// of a tensor that was kept in 1x128 tiles,
//   v[r][c] = code * scale_inv * row[r] * col[c],   v^T quantized in 1x128 tiles.
// With row = rstd and col = gamma it is the normalised tensor recomputed from
// the checkpoint of the norm's input.  FP32 products, one rounding.
//
// HBM-bound: one byte in, one byte out per element.
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
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kTileK, r0 = static_cast<int64_t>(blockIdx.y) * kTileK;
  const int c = 4 * (threadIdx.x % 32), r = kRegRows * (threadIdx.x / 32);
  const int ncols = left(a.cols - c0) < kTileK ? left(a.cols - c0) : kTileK, nrows = left(a.rows - r0);
  const uint8_t* q = a.x.q + (r0 + r) * a.x.ldq + c0;
  const float* s = a.x.s + c0 / kTileK * a.x.lds + r0 + r;
  float v[1][kRegRows][kRegCols], col[4];
  load_cols<4>(elem_of(a.ct, a.col, a.col ? c0 : 0), a.ct, c, ncols, col);
#pragma unroll
  for (int i = 0; i < kRegRows; ++i) {
    uint32_t w[1] = {0u};
    float f = 0.0f;
    if (r + i < nrows) {
      load_codes<4>(q + i * a.x.ldq, c, ncols, w);
      f = s[i];
    }
    decode<4>(a.x.type, w, f, v[0][i]);
    if (a.row) {
      f = r + i < nrows ? a.row[r0 + r + i] : 0.0f;
#pragma unroll
      for (int j = 0; j < kRegCols; ++j) v[0][i][j] *= f;
    }
    if (a.col) {
#pragma unroll
      for (int j = 0; j < kRegCols; ++j) v[0][i][j] *= col[j];
    }
  }
  const amp_fp8_tiles o[1] = {a.qt};
  const int64_t first[1] = {c0};
  store_regions_t<1>(l, o, first, r0, a.rows, ncols, v);
}

}  // namespace

hipError_t launch_requantize(const amp_fp8_tiles& x, int64_t rows, int64_t cols, const float* row, const void* col, int ct,
                             const amp_fp8_tiles& qt, hipStream_t s) {
  constexpr int64_t kMost = 65535 * static_cast<int64_t>(kTileK);   // rows a launch: the grid's y bound
  for (int64_t r0 = 0; r0 < rows; r0 += kMost) {
    RequantArgs a{x, qt, rows - r0 < kMost ? rows - r0 : kMost, cols, row ? row + r0 : nullptr, col, ct};
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
