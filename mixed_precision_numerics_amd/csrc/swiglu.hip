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

// One vector of R rows (S apart, from row0 on) in 1x128 tiles; `blk` is the
// tile's index along K.  Lane i of a tile's lane group stores row i's scale.
template <int E, int R, bool FULL>
__device__ __forceinline__ void store_row_tiles(const amp_fp8_tiles& o, int64_t row0, int S, int64_t rows, int64_t c0, int c,
                                                int n, int64_t blk, float (&v)[R][E]) {
  constexpr int G = kTileK / E;
  uint32_t m[R], top = 0, w[R][E / 4];
  float sc[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = group_max<G>(mag(abs_max<E>(0.0f, v[i])));
    top = top > m[i] ? top : m[i];
  }
  const float inv = tile_scales<R>(m, fp8_max(o.type), sc);
  const int64_t mine = row0 + (threadIdx.x & 3) * S;
  if (threadIdx.x % G < R && mine < rows && (FULL || c / kTileK * kTileK < n)) o.s[blk * o.lds + mine] = inv;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int k = 0; k < E; ++k) v[i][k] *= sc[i];
  encode<R, E, false>(o.type, v, top >= kInfBits, w);
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (row0 + i * S < rows) store_codes<E, FULL>(o.q + (row0 + i * S) * o.ldq + c0, c, n, w[i]);
}

// W threads cover W vectors of a row, 256 / W rows side by side and R of
// those groups one after the other; blockIdx.x runs along the row.  FULL: the
// row is whole spans of W vectors.
template <int XT, int W, int R, bool FULL>
__global__ __launch_bounds__(256) void swiglu_rows(const GateArgs a) {
  constexpr int E = kVec<XT>, S = 256 / W;
  __shared__ uint32_t redm[256 / kWave];
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * (W * E);   // the block's first column
  const int c = threadIdx.x % W * E, n = left(a.cols - c0);
  const int sub = W >= kWave ? __builtin_amdgcn_readfirstlane(threadIdx.x / W) : threadIdx.x / W;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * (S * R) + sub;
  const float scale = a.scale ? *a.scale : 1.0f;
  const uint32_t seen = amax_seen(a.amax);
  u32x4 wg[R], wu[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + i * S;
    wg[i] = wu[i] = u32x4{0u, 0u, 0u, 0u};
    if (row < a.rows) {
      const void* p = elem<XT>(a.x, row * a.ldx + c0);
      wg[i] = load_vec<XT, FULL>(p, c, n);
      wu[i] = load_vec<XT, FULL>(elem<XT>(p, a.cols), c, n);
    }
  }
  float y[R][E], am = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float g[E], u[E];
    widen<XT>(wg[i], g);
    widen<XT>(wu[i], u);
#pragma unroll
    for (int k = 0; k < E; ++k) y[i][k] = g[k] * gate(g[k]).s * u[k];
    am = abs_max<E>(am, y[i]);
  }
  if (a.y) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = row0 + i * S, at = (row * a.ldy + c0) * (a.yt == AMP_F16 || a.yt == AMP_BF16 ? 2 : 1);
      store_plain<1, E, FULL>(static_cast<uint8_t*>(a.y) + at, a.yt, c, 0, n, row < a.rows, scale, am,
                              reinterpret_cast<const float(&)[1][E]>(y[i]));
    }
  }
  if (a.yq.q) store_row_tiles<E, R, FULL>(a.yq, row0, S, a.rows, c0, c, n, (c0 + c) / kTileK, y);
  if (a.ck.q) {
#pragma unroll
    for (int i = 0; i < R; ++i) widen<XT>(wg[i], y[i]);
    store_row_tiles<E, R, FULL>(a.ck, row0, S, a.rows, c0, c, n, tile_of(c0 + c, 0, a.cols), y);
#pragma unroll
    for (int i = 0; i < R; ++i) widen<XT>(wu[i], y[i]);
    amp_fp8_tiles up = a.ck;
    up.q += a.cols;
    store_row_tiles<E, R, FULL>(up, row0, S, a.rows, c0, c, n, tile_of(c0 + c, 1, a.cols), y);
  }
  if (a.amax) block_amax(am, seen, redm, a.amax);
}

// Backward with dx in the gradient's own type only: element-wise, laid out
// as above.
template <int XT, bool CK, int W, int R, bool FULL>
__global__ __launch_bounds__(256) void swiglu_back_rows(const GateArgs a) {
  constexpr int E = kVec<XT>, S = 256 / W;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * (W * E);
  const int c = threadIdx.x % W * E, n = left(a.cols - c0);
  const int sub = W >= kWave ? __builtin_amdgcn_readfirstlane(threadIdx.x / W) : threadIdx.x / W;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * (S * R) + sub;
  if (!FULL && c >= n) return;
  u32x4 wd[R], wg[R], wu[R];
  uint32_t qg[R][E / 4], qu[R][E / 4];
  float sg[R], su[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + i * S < a.rows ? row0 + i * S : a.rows - 1;   // read again, not used
    wd[i] = load_vec<XT, FULL>(elem<XT>(a.dy, row * a.lddy + c0), c, n);
    if constexpr (CK) {
      const uint8_t* q = a.ck.q + row * a.ck.ldq + c0;
      load_codes<E, FULL>(q, c, n, qg[i]);
      load_codes<E, FULL>(q + a.cols, c, n, qu[i]);
      sg[i] = a.ck.s[tile_of(c0 + c, 0, a.cols) * a.ck.lds + row];
      su[i] = a.ck.s[tile_of(c0 + c, 1, a.cols) * a.ck.lds + row];
    } else {
      const void* p = elem<XT>(a.x, row * a.ldx + c0);
      wg[i] = load_vec<XT, FULL>(p, c, n);
      wu[i] = load_vec<XT, FULL>(elem<XT>(p, a.cols), c, n);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + i * S;
    if (row >= a.rows) return;
    float g[E], u[E], dy[E], dg[E], du[E];
    widen<XT>(wd[i], dy);
    if constexpr (CK) {
      decode<E>(a.ck.type, qg[i], sg[i], g);
      decode<E>(a.ck.type, qu[i], su[i], u);
    } else {
      widen<XT>(wg[i], g);
      widen<XT>(wu[i], u);
    }
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const Gate p = gate(g[k]);
      const float t = dy[k] * p.s;
      du[k] = t * g[k];
      dg[k] = t * u[k] * (1.0f + g[k] * p.om);
    }
    void* p = elem<XT>(a.y, row * a.ldy + c0);
    store_vec<XT, FULL>(p, c, n, narrow<XT>(dg));
    store_vec<XT, FULL>(elem<XT>(p, a.cols), c, n, narrow<XT>(du));
  }
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
  const int c = 4 * cg, r = kRegRows * rg;
  const int ncols = left(a.cols - c0) < kTileK ? left(a.cols - c0) : kTileK, nrows = left(a.rows - r0);
  float v[3][kRegRows][kRegCols];   // dg, du, y
#pragma unroll
  for (int i = 0; i < kRegRows; ++i) {
    const int64_t row = r0 + r + i;
    float g[4] = {}, u[4] = {}, dy[4] = {};
    if (r + i < nrows) {
      load_cols<4>(elem<XT>(a.dy, row * a.lddy + c0), XT, c, ncols, dy);
      if constexpr (CK) {
        uint32_t q[1];
        load_codes<4>(a.ck.q + row * a.ck.ldq + c0, c, ncols, q);
        decode<4>(a.ck.type, q, a.ck.s[tile_of(c0, 0, a.cols) * a.ck.lds + row], g);
        load_codes<4>(a.ck.q + row * a.ck.ldq + a.cols + c0, c, ncols, q);
        decode<4>(a.ck.type, q, a.ck.s[tile_of(c0, 1, a.cols) * a.ck.lds + row], u);
      } else {
        load_cols<4>(elem<XT>(a.x, row * a.ldx + c0), XT, c, ncols, g);
        load_cols<4>(elem<XT>(a.x, row * a.ldx + a.cols + c0), XT, c, ncols, u);
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
    if (a.y && r + i < nrows) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        void* p = elem<XT>(a.y, row * a.ldy + (n ? a.cols : 0) + c0);
        const float(&f)[4] = v[n][i];
        if constexpr (XT == AMP_F32) {
          store_vec<AMP_F32>(p, c, ncols, narrow<AMP_F32>(f));
        } else {
          const uint32_t h[2] = {pack16(XT == AMP_BF16, f[0], f[1]), pack16(XT == AMP_BF16, f[2], f[3])};
          store16<2>(p, c, ncols, h);
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
        if (cg == 0) rmax[n][r + i] = m;
      }
    __syncthreads();
    if (t < 2 * kTileK) {
      const int n = t / kTileK, i = t % kTileK;
      const uint32_t m = rmax[n][i];
      const float sc = scale_of(m, fp8_max(a.dxq.type));
      rscale[n][i] = m >= kInfBits ? -sc : sc;   // sign: the tile holds a NaN or infinity
      if (i < nrows) a.dxq.s[tile_of(c0, n, a.cols) * a.dxq.lds + r0 + i] = 1.0f / sc;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < kRegRows; ++i) {
        const float sc = rscale[n][r + i];
        float f[1][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) f[0][k] = v[n][i][k] * fabsf(sc);
        uint32_t w[1][1];
        encode<1, 4, false>(a.dxq.type, f, sc < 0.0f, w);
        if (r + i < nrows) store_codes<4>(a.dxq.q + (r0 + r + i) * a.dxq.ldq + (n ? a.cols : 0) + c0, c, ncols, w[0]);
      }
  }
  if (a.dxqt.q || a.yqt.q) {
    const amp_fp8_tiles o[3] = {a.dxqt, a.dxqt, a.yqt};
    const int64_t first[3] = {c0, a.cols + c0, c0};
    store_regions_t<3>(l, o, first, r0, a.rows, ncols, v);
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

// Calls f(first row, rows) for slices of at most `most` rows.
template <typename F>
hipError_t in_slices(int64_t rows, int64_t most, F f) {
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    f(r0, rows - r0 < most ? rows - r0 : most);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

constexpr int kGridY = 65535;

template <int XT, int W, int R>
hipError_t run_swiglu(const GateArgs& whole, hipStream_t s) {
  constexpr int E = kVec<XT>, per = 256 / W * R;
  const bool full = whole.cols % (W * E) == 0;
  return in_slices(whole.rows, static_cast<int64_t>(kGridY) * per, [&](int64_t r0, int64_t rows) {
    GateArgs a = whole;
    a.rows = rows;
    a.x = elem<XT>(a.x, r0 * a.ldx);
    if (a.y) a.y = static_cast<uint8_t*>(a.y) + r0 * a.ldy * dtype_bytes(a.yt);
    if (a.yq.q) { a.yq.q += r0 * a.yq.ldq; a.yq.s += r0; }
    if (a.ck.q) { a.ck.q += r0 * a.ck.ldq; a.ck.s += r0; }
    const dim3 grid(static_cast<unsigned>((a.cols + W * E - 1) / (W * E)), static_cast<unsigned>((rows + per - 1) / per));
    if (full) swiglu_rows<XT, W, R, true><<<grid, 256, 0, s>>>(a);
    else swiglu_rows<XT, W, R, false><<<grid, 256, 0, s>>>(a);
  });
}

template <int XT>
hipError_t dispatch_swiglu(const GateArgs& a, hipStream_t s) {
  switch (row_width(a.cols, kVec<XT>)) {
    case 256: return run_swiglu<XT, 256, 2>(a, s);
    case 64: return run_swiglu<XT, 64, 2>(a, s);
    default: return run_swiglu<XT, 32, 2>(a, s);
  }
}

template <int XT, bool CK, int W, int R>
hipError_t run_swiglu_back(const GateArgs& whole, hipStream_t s) {
  constexpr int E = kVec<XT>, per = 256 / W * R;
  const bool full = whole.cols % (W * E) == 0;
  return in_slices(whole.rows, static_cast<int64_t>(kGridY) * per, [&](int64_t r0, int64_t rows) {
    GateArgs a = whole;
    a.rows = rows;
    a.dy = elem<XT>(a.dy, r0 * a.lddy);
    a.y = elem<XT>(a.y, r0 * a.ldy);
    if (CK) { a.ck.q += r0 * a.ck.ldq; a.ck.s += r0; }
    else a.x = elem<XT>(a.x, r0 * a.ldx);
    const dim3 grid(static_cast<unsigned>((a.cols + W * E - 1) / (W * E)), static_cast<unsigned>((rows + per - 1) / per));
    if (full) swiglu_back_rows<XT, CK, W, R, true><<<grid, 256, 0, s>>>(a);
    else swiglu_back_rows<XT, CK, W, R, false><<<grid, 256, 0, s>>>(a);
  });
}

template <int XT, bool CK>
hipError_t dispatch_swiglu_back(const GateArgs& whole, hipStream_t s) {
  if (whole.dxq.q || whole.dxqt.q || whole.yqt.q) {
    return in_slices(whole.rows, static_cast<int64_t>(kGridY) * kTileK, [&](int64_t r0, int64_t rows) {
      GateArgs a = whole;
      a.rows = rows;
      a.dy = elem<XT>(a.dy, r0 * a.lddy);
      if (a.y) a.y = elem<XT>(a.y, r0 * a.ldy);
      if (CK) { a.ck.q += r0 * a.ck.ldq; a.ck.s += r0; }
      else a.x = elem<XT>(a.x, r0 * a.ldx);
      if (a.dxq.q) { a.dxq.q += r0 * a.dxq.ldq; a.dxq.s += r0; }
      if (a.dxqt.q) { a.dxqt.q += r0; a.dxqt.s += r0 / kTileK * a.dxqt.lds; }
      if (a.yqt.q) { a.yqt.q += r0; a.yqt.s += r0 / kTileK * a.yqt.lds; }
      const dim3 grid(static_cast<unsigned>((a.cols + kTileK - 1) / kTileK), static_cast<unsigned>((rows + kTileK - 1) / kTileK));
      swiglu_back_region<XT, CK><<<grid, kRegThreads, 0, s>>>(a);
    });
  }
  switch (row_width(whole.cols, kVec<XT>)) {
    case 256: return run_swiglu_back<XT, CK, 256, 2>(whole, s);
    case 64: return run_swiglu_back<XT, CK, 64, 2>(whole, s);
    default: return run_swiglu_back<XT, CK, 32, 2>(whole, s);
  }
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
