// Gated activation with 16-bit or FP8 outputs, and its backward pass from the
// stored input or from an FP8 checkpoint (gfx950).
//
//   x = [g | u],  s = 1 / (1 + exp(-g)),  y = g s u
//   du = dy g s,  dg = dy u s (1 + g (1 - s))
//
// FP32 arithmetic, one rounding per output.  With e = exp(-g) the factor
// 1 - s is e s, which keeps its relative precision where s is near 1.
#include "tiles.hpp"

namespace amp {
namespace {

struct GateArgs {
  const void* x; int64_t ldx;
  const void* dy; int64_t lddy;
  void* y; int yt; int64_t ldy;
  const float* scale; float* amax;
  amp_fp8_tiles yq, ck;          // forward: outputs; backward: ck is the input
  amp_fp8_tiles dxq, dxqt, yqt;  // backward
  int64_t rows, cols;
};

template <int XT>
__device__ __forceinline__ int64_t elem_bytes(int64_t i) { return i * (XT == AMP_F32 ? 4 : 2); }
template <int XT>
__device__ __forceinline__ const void* at(const void* p, int64_t i) { return static_cast<const uint8_t*>(p) + elem_bytes<XT>(i); }
template <int XT>
__device__ __forceinline__ void* at(void* p, int64_t i) { return static_cast<uint8_t*>(p) + elem_bytes<XT>(i); }

// s = 1 / (1 + e), e = exp(-g), from the hardware's exponential and
// reciprocal (each within an ulp; the scaled argument adds |g| 2^-24, so s is
// good to a few 2^-23 over the range where it is not negligible).  g = -inf
// gives s = 0 and, as in the formula, 0 * inf = NaN for g s.
struct Gate { float s, om; };   // s and 1 - s
__device__ __forceinline__ Gate gate(float g) {
  const float e = __builtin_amdgcn_exp2f(g * -1.4426950408889634f);
  const float s = __builtin_amdgcn_rcpf(1.0f + e);
  return {s, e > 1.7e38f ? 1.0f : e * s};
}

// Index along K of the tile that holds column c of half `half`: the tiles
// start again at the second half.
__device__ __forceinline__ int64_t tile_of(int64_t c, int half, int64_t cols) {
  return c / kTileK + (half ? (cols + kTileK - 1) / kTileK : 0);
}

// W threads cover W vectors of a row, 256 / W rows side by side and R of
// those groups one after the other; blockIdx.x runs along the row.
template <int XT, int W, int R>
__global__ __launch_bounds__(256) void swiglu_rows(const GateArgs a) {
  constexpr int E = kVec<XT>, S = 256 / W;
  __shared__ uint32_t redm[256 / kWave];
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * W + threadIdx.x % W) * E;
  const float scale = a.scale ? *a.scale : 1.0f;
  float am = 0.0f;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * (S * R); r0 < a.rows; r0 += static_cast<int64_t>(gridDim.y) * (S * R)) {
    u32x4 wg[R], wu[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = r0 + i * S + threadIdx.x / W;
      wg[i] = wu[i] = u32x4{0u, 0u, 0u, 0u};
      if (row < a.rows) {
        wg[i] = load_vec<XT>(at<XT>(a.x, row * a.ldx), c, a.cols);
        wu[i] = load_vec<XT>(at<XT>(a.x, row * a.ldx + a.cols), c, a.cols);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = r0 + i * S + threadIdx.x / W;
      const bool live = row < a.rows;
      float g[E], u[E], y[E];
      widen<XT>(wg[i], g);
      widen<XT>(wu[i], u);
#pragma unroll
      for (int k = 0; k < E; ++k) y[k] = g[k] * gate(g[k]).s * u[k];
      const float m = abs_max<E>(0.0f, y);
      am = __builtin_elementwise_maximum(am, m);
      if (a.yq.q) store_tile<E>(a.yq, row, c, a.cols, c / kTileK, live, y);
      if (a.ck.q) {
        store_tile<E>(a.ck, row, c, a.cols, tile_of(c, 0, a.cols), live, g);
        amp_fp8_tiles up = a.ck;
        up.q += a.cols;
        store_tile<E>(up, row, c, a.cols, tile_of(c, 1, a.cols), live, u);
      }
      if (a.y && live) store_plain<E>(a.y, a.yt, row * a.ldy, c, a.cols, scale, m, y);
    }
  }
  if (a.amax) {
    const uint32_t m = block_max_u32<256>(mag(am), redm);
    if (threadIdx.x == 0 && m != 0) amax_update(a.amax, m);
  }
}

// Backward with dx in the gradient's own type only: element-wise, as above.
template <int XT, bool CK, int W, int R>
__global__ __launch_bounds__(256) void swiglu_back_rows(const GateArgs a) {
  constexpr int E = kVec<XT>, S = 256 / W;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * W + threadIdx.x % W) * E;
  if (c >= a.cols) return;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * (S * R); r0 < a.rows; r0 += static_cast<int64_t>(gridDim.y) * (S * R)) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = r0 + i * S + threadIdx.x / W;
      if (row >= a.rows) continue;
      float g[E], u[E], dy[E], dg[E], du[E];
      widen<XT>(load_vec<XT>(at<XT>(a.dy, row * a.lddy), c, a.cols), dy);
      if constexpr (CK) {
        uint32_t q[E / 4];
        load_codes<E>(a.ck.q + row * a.ck.ldq, c, a.cols, q);
        decode<E>(a.ck.type, q, a.ck.s[tile_of(c, 0, a.cols) * a.ck.lds + row], g);
        load_codes<E>(a.ck.q + row * a.ck.ldq + a.cols, c, a.cols, q);
        decode<E>(a.ck.type, q, a.ck.s[tile_of(c, 1, a.cols) * a.ck.lds + row], u);
      } else {
        widen<XT>(load_vec<XT>(at<XT>(a.x, row * a.ldx), c, a.cols), g);
        widen<XT>(load_vec<XT>(at<XT>(a.x, row * a.ldx + a.cols), c, a.cols), u);
      }
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const Gate p = gate(g[k]);
        const float t = dy[k] * p.s;
        du[k] = t * g[k];
        dg[k] = t * u[k] * (1.0f + g[k] * p.om);
      }
      store_vec<XT>(at<XT>(a.y, row * a.ldy), c, a.cols, narrow<XT>(dg));
      store_vec<XT>(at<XT>(a.y, row * a.ldy + a.cols), c, a.cols, narrow<XT>(du));
    }
  }
}

// 4 elements of a row of the type XT.
template <int XT>
__device__ __forceinline__ void load4(const void* p, int64_t c, int64_t cols, float (&v)[4]) {
  load_cols<4>(p, XT, c, cols, v);
}

// Backward with FP8 operands: one 128x128 region of dy, g and u per block.
// dg, du and y are formed once in registers and leave from there in every
// form asked for: dx in dy's type, dx in row tiles (dgrad), dx^T and y^T in
// tiles along the rows (wgrad).
template <int XT, bool CK>
__global__ __launch_bounds__(kRegThreads) void swiglu_back_region(const GateArgs a) {
  __shared__ RegLds<3> l;
  __shared__ uint32_t rmax[2][kTileK];
  __shared__ float rscale[2][kTileK];
  const int t = threadIdx.x, cg = t % 32, rg = t / 32;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kTileK, r0 = static_cast<int64_t>(blockIdx.y) * kTileK;
  const int64_t c = c0 + 4 * cg, r = r0 + kRegRows * rg;
  float v[3][kRegRows][kRegCols];   // dg, du, y
#pragma unroll
  for (int i = 0; i < kRegRows; ++i) {
    const int64_t row = r + i;
    float g[4] = {}, u[4] = {}, dy[4] = {};
    if (row < a.rows) {
      load4<XT>(at<XT>(a.dy, row * a.lddy), c, a.cols, dy);
      if constexpr (CK) {
        uint32_t q[1];
        load_codes<4>(a.ck.q + row * a.ck.ldq, c, a.cols, q);
        decode<4>(a.ck.type, q, a.ck.s[tile_of(c0, 0, a.cols) * a.ck.lds + row], g);
        load_codes<4>(a.ck.q + row * a.ck.ldq + a.cols, c, a.cols, q);
        decode<4>(a.ck.type, q, a.ck.s[tile_of(c0, 1, a.cols) * a.ck.lds + row], u);
      } else {
        load4<XT>(at<XT>(a.x, row * a.ldx), c, a.cols, g);
        load4<XT>(at<XT>(a.x, row * a.ldx + a.cols), c, a.cols, u);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Gate p = gate(g[k]);
      const float d = dy[k] * p.s, gu = g[k] * p.s;
      v[0][i][k] = d * u[k] * (1.0f + g[k] * p.om);
      v[1][i][k] = d * g[k];
      v[2][i][k] = gu * u[k];
    }
    if (a.y && row < a.rows) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float f[4] = {v[n][i][0], v[n][i][1], v[n][i][2], v[n][i][3]};
        const int64_t base = row * a.ldy + (n ? a.cols : 0);
        if constexpr (XT == AMP_F32) {
          store_vec<AMP_F32>(at<XT>(a.y, base), c, a.cols, narrow<AMP_F32>(f));
        } else {
          store_plain<4>(a.y, XT, base, c, a.cols, 1.0f, 0.0f, f);
        }
      }
    }
  }
  if (a.dxq.q) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < kRegRows; ++i) {
        const uint32_t m = group_max<32>(mag(abs_max<4>(0.0f, v[n][i])));
        if (cg == 0) rmax[n][kRegRows * rg + i] = m;
      }
    __syncthreads();
    if (t < 2 * kTileK) {
      const int n = t / kTileK, i = t % kTileK;
      const uint32_t m = rmax[n][i];
      const float sc = scale_of(m, fp8_max(a.dxq.type));
      rscale[n][i] = m >= 0x7f800000u ? -sc : sc;   // sign: the tile holds a NaN or infinity
      if (r0 + i < a.rows) a.dxq.s[tile_of(c0, n, a.cols) * a.dxq.lds + r0 + i] = 1.0f / sc;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < kRegRows; ++i) {
        const float sc = rscale[n][kRegRows * rg + i];
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = v[n][i][k] * fabsf(sc);
        uint32_t w[1];
        encode<4>(a.dxq.type, f, sc < 0.0f, w);
        if (r + i < a.rows) store_codes<4>(a.dxq.q + (r + i) * a.dxq.ldq + (n ? a.cols : 0), c, a.cols, w);
      }
  }
  if (a.dxqt.q || a.yqt.q) {
    const amp_fp8_tiles o[3] = {a.dxqt, a.dxqt, a.yqt};
    const int64_t first[3] = {c0, a.cols + c0, c0};
    store_regions_t<3>(l, o, first, r0, a.rows, static_cast<int>(a.cols - c0 < kTileK ? a.cols - c0 : kTileK), v);
  }
}

// The widest W whose whole vectors overshoot the row by at most an eighth
// (a tile's lanes stay together in every case).
int row_width(int64_t cols, int e) {
  for (int w : {256, 64}) {
    const int64_t span = static_cast<int64_t>(w) * e;
    if ((cols + span - 1) / span * span * 8 <= cols * 9) return w;
  }
  return 32;
}

dim3 row_grid(int64_t rows, int64_t cols, int w, int e, int per) {
  const int64_t x = (cols + w * e - 1) / (w * e);
  int64_t y = (rows + per - 1) / per;
  if (y > 65535) y = 65535;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
}

template <int XT>
hipError_t dispatch_swiglu(const GateArgs& a, hipStream_t s) {
  constexpr int E = kVec<XT>, R = 2;
  const int w = row_width(a.cols, E);
  const dim3 grid = row_grid(a.rows, a.cols, w, E, 256 / w * R);
  if (w == 256) swiglu_rows<XT, 256, R><<<grid, 256, 0, s>>>(a);
  else if (w == 64) swiglu_rows<XT, 64, R><<<grid, 256, 0, s>>>(a);
  else swiglu_rows<XT, 32, R><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int XT, bool CK>
hipError_t dispatch_swiglu_back(const GateArgs& a, hipStream_t s) {
  if (a.dxq.q || a.dxqt.q || a.yqt.q) {
    const dim3 grid(static_cast<unsigned>((a.cols + kTileK - 1) / kTileK), static_cast<unsigned>((a.rows + kTileK - 1) / kTileK));
    swiglu_back_region<XT, CK><<<grid, kRegThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  constexpr int E = kVec<XT>, R = 2;
  const int w = row_width(a.cols, E);
  const dim3 grid = row_grid(a.rows, a.cols, w, E, 256 / w * R);
  if (w == 256) swiglu_back_rows<XT, CK, 256, R><<<grid, 256, 0, s>>>(a);
  else if (w == 64) swiglu_back_rows<XT, CK, 64, R><<<grid, 256, 0, s>>>(a);
  else swiglu_back_rows<XT, CK, 32, R><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int XT>
hipError_t dispatch_swiglu_back_x(const GateArgs& a, hipStream_t s) {
  return a.ck.q ? dispatch_swiglu_back<XT, true>(a, s) : dispatch_swiglu_back<XT, false>(a, s);
}

}  // namespace

hipError_t launch_swiglu(const void* x, int xt, int64_t rows, int64_t cols, int64_t ldx, void* y, int yt, int64_t ldy,
                         const float* scale, float* amax, const amp_fp8_tiles& yq, const amp_fp8_tiles& ckpt, hipStream_t s) {
  GateArgs a{};
  a.x = x; a.ldx = ldx; a.y = y; a.yt = yt; a.ldy = ldy; a.scale = scale; a.amax = amax;
  a.yq = yq; a.ck = ckpt; a.rows = rows; a.cols = cols;
  switch (xt) {
    case AMP_F32: return dispatch_swiglu<AMP_F32>(a, s);
    case AMP_BF16: return dispatch_swiglu<AMP_BF16>(a, s);
    default: return dispatch_swiglu<AMP_F16>(a, s);
  }
}

hipError_t launch_swiglu_backward(const void* dy, int dt, int64_t rows, int64_t cols, int64_t lddy, const void* x, int64_t ldx,
                                  const amp_fp8_tiles& ckpt, void* dx, int64_t lddx, const amp_fp8_tiles& dxq,
                                  const amp_fp8_tiles& dxqt, const amp_fp8_tiles& yqt, hipStream_t s) {
  GateArgs a{};
  a.x = x; a.ldx = ldx; a.dy = dy; a.lddy = lddy; a.y = dx; a.ldy = lddx;
  a.ck = ckpt; a.dxq = dxq; a.dxqt = dxqt; a.yqt = yqt; a.rows = rows; a.cols = cols;
  switch (dt) {
    case AMP_F32: return dispatch_swiglu_back_x<AMP_F32>(a, s);
    case AMP_BF16: return dispatch_swiglu_back_x<AMP_BF16>(a, s);
    default: return dispatch_swiglu_back_x<AMP_F16>(a, s);
  }
}

}  // namespace amp
