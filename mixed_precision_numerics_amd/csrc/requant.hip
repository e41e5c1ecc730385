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
  const int64_t c = c0 + 4 * (threadIdx.x % 32), r = r0 + kRegRows * (threadIdx.x / 32);
  float v[1][kRegRows][kRegCols], col[4];
  load_cols<4>(a.col, a.ct, c, a.cols, col);
#pragma unroll
  for (int i = 0; i < kRegRows; ++i) {
    uint32_t w[1] = {0u};
    float s = 0.0f;
    if (r + i < a.rows) {
      load_codes<4>(a.x.q + (r + i) * a.x.ldq, c, a.cols, w);
      s = a.x.s[c0 / kTileK * a.x.lds + r + i];
    }
    decode<4>(a.x.type, w, s, v[0][i]);
    if (a.row) {
      const float f = r + i < a.rows ? a.row[r + i] : 0.0f;
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
  store_regions_t<1>(l, o, first, r0, a.rows, static_cast<int>(a.cols - c0 < kTileK ? a.cols - c0 : kTileK), v);
}

}  // namespace

hipError_t launch_requantize(const amp_fp8_tiles& x, int64_t rows, int64_t cols, const float* row, const void* col, int ct,
                             const amp_fp8_tiles& qt, hipStream_t s) {
  const RequantArgs a{x, qt, rows, cols, row, col, ct};
  const dim3 grid(static_cast<unsigned>((cols + kTileK - 1) / kTileK), static_cast<unsigned>((rows + kTileK - 1) / kTileK));
  requant_region<<<grid, kRegThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace amp
